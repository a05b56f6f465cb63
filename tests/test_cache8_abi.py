"""The rotation and the 8-bit cache reject bad arguments on the host, before any CUDA call (no GPU needed)."""

import pytest
import torch

from io_aware_exact_04_gb300 import _lib, api
from tests.cache8_ref import least

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
A, M = 0x10000, 0x10008  # 16-byte aligned and misaligned fake addresses: never dereferenced


@pytest.fixture(scope="module")
def lib(built):
    return _lib.load("libfa.so")


def rows(data=A, st=1024, sh=64):
    return _lib.Rows(data, st, sh)


def pages(**kw):
    x = dict(k=A, v=A, page_stride=4096, head_stride=1024, token_stride=64, n_pages=8, page_size=64, table=A,
             table_stride=4, table_width=4)
    x.update(kw)
    return _lib.Pages(*x.values())


def scales(**kw):
    x = dict(k=A, v=A, page_stride=4, head_stride=2, block=32)
    x.update(kw)
    return _lib.Scales(*x.values())


def angles(**kw):
    x = dict(angles=A, row_stride=64, positions=100, dim=64, interleaved=0, at=None)
    x.update(kw)
    return _lib.Rotary(*x.values())


def tree(lib, q=None, k=None, v=None, o=None, lse=A, cache=None, sc=None, lens=A, cu=A, mask=None, words=0, B=1, T=4,
         Hq=4, Hkv=2, d=64, dtype=0, scale=0.125, ws=A, nbytes=1 << 40):
    q, k, v, o = (rows() if x is None else x for x in (q, k, v, o))
    return lib.fa_forward_tree_8bit(q, k, v, o, lse, cache or pages(), sc or scales(), lens, cu, mask, words, B, T, Hq, Hkv,
                                    d, dtype, scale, ws, nbytes, None)


def append(lib, k=None, v=None, cache=None, sc=None, start=A, cu=A, pick=None, B=1, T=4, Tkv=4, Hkv=2, d=64, dtype=0):
    k, v = (rows() if x is None else x for x in (k, v))
    return lib.fa_cache_append_8bit(k, v, cache or pages(), sc or scales(), start, cu, pick, B, T, Tkv, Hkv, d, dtype, None)


def rotary(lib, q=0, k=0, v=0, qo=0, ko=0, cache=0, sc=0, turn=0, start=A, cu=A, B=1, T=4, Hq=4, Hkv=2, d=64, dtype=0):
    q, k, v, qo, ko = (rows() if x == 0 else x for x in (q, k, v, qo, ko))
    cache, sc, turn = (make() if x == 0 else x for x, make in ((cache, pages), (sc, scales), (turn, angles)))
    return lib.fa_rotary_append(q, k, v, qo, ko, cache, sc, turn, start, cu, B, T, Hq, Hkv, d, dtype, None)


@pytest.mark.parametrize("call", [tree, append, rotary])
def test_sizes_pages_and_scales(lib, call):
    for d in (0, 32, 96, 256):
        assert call(lib, d=d) == UNSUPPORTED
    for kw in (dict(B=-1), dict(T=-1), dict(Hkv=0), dict(dtype=2), dict(cu=None)):
        assert call(lib, **kw) == INVALID, kw
    for kw in (dict(B=(1 << 20) + 1), dict(T=(1 << 30) + 1, **({"Tkv": (1 << 30) + 1} if call is append else {}))):
        assert call(lib, **kw) == UNSUPPORTED, kw
    for kw in (dict(k=None), dict(v=None), dict(table=None), dict(n_pages=0), dict(table_width=0), dict(table_stride=3),
               dict(page_stride=0), dict(head_stride=-16), dict(token_stride=72)):
        assert call(lib, cache=pages(**kw)) == INVALID, kw
    for kw in (dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(table_width=1 << 27, table_stride=1 << 27)):
        assert call(lib, cache=pages(**kw)) == UNSUPPORTED, kw
    for kw in (dict(k=M), dict(v=M)):
        assert call(lib, cache=pages(**kw)) == MISALIGNED, kw
    for kw in (dict(k=None), dict(v=None), dict(page_stride=0), dict(head_stride=-1)):
        assert call(lib, sc=scales(**kw)) == INVALID, kw
    for kw in (dict(block=8), dict(block=48), dict(block=128)):  # 128: more than a page
        assert call(lib, sc=scales(**kw)) == UNSUPPORTED, kw
    for kw in (dict(k=A + 2), dict(v=A + 1)):
        assert call(lib, sc=scales(**kw)) == MISALIGNED, kw
    for name in ("k", "v"):
        assert call(lib, **{name: rows(data=None)}) == INVALID
        assert call(lib, **{name: rows(data=M)}) == MISALIGNED
        for bad in (dict(st=0), dict(st=-64), dict(st=12), dict(sh=0), dict(sh=-8), dict(sh=63)):
            assert call(lib, **{name: rows(**bad)}) == INVALID, bad
    assert call(lib, T=0, **({"Tkv": 0} if call is append else {})) == OK
    assert call(lib, B=0) == OK


def test_tree_argument_errors(lib):
    for kw in (dict(scale=0.0), dict(scale=float("nan")), dict(Hq=5), dict(lens=None), dict(ws=None), dict(mask=A, words=0)):
        assert tree(lib, **kw) == INVALID, kw
    assert tree(lib, Hq=129, Hkv=1) == UNSUPPORTED
    assert tree(lib, mask=A, words=(1 << 20) + 1) == UNSUPPORTED
    assert tree(lib, ws=A + 16) == MISALIGNED
    assert tree(lib, lse=M) == MISALIGNED
    assert lib.fa_forward_tree_8bit_workspace_size(96) == 0


def test_append_argument_errors(lib):
    assert append(lib, T=4, Tkv=5) == INVALID
    assert append(lib, pick=A, Tkv=0) == INVALID
    assert append(lib, pick=A, Tkv=-1) == INVALID
    assert append(lib, start=None) == INVALID


def test_rotary_argument_errors(lib):
    for kw in (dict(angles=None), dict(positions=0), dict(dim=0), dict(dim=24), dict(dim=80), dict(interleaved=2),
               dict(row_stride=60), dict(row_stride=66)):
        assert rotary(lib, turn=angles(**kw)) == INVALID, kw
    assert rotary(lib, turn=angles(angles=M)) == MISALIGNED
    assert rotary(lib, turn=None) == INVALID
    assert rotary(lib, q=None) == INVALID and rotary(lib, qo=None) == INVALID
    assert rotary(lib, qo=rows(data=M)) == MISALIGNED and rotary(lib, ko=rows(st=12)) == INVALID
    assert rotary(lib, Hq=5) == INVALID and rotary(lib, start=None) == INVALID
    # without a cache the positions have to be given, and something to be written
    assert rotary(lib, cache=None) == INVALID
    assert rotary(lib, cache=None, q=None, qo=None, ko=None, turn=angles(at=A)) == INVALID


def test_pool_argument_errors(lib):
    def pool(**kw):
        x = dict(data=A, plane_stride=1 << 20, planes=2, n_pages=8, Hkv=2, page_size=64, d=64, table=A, lens=A, slots=4,
                 table_width=4)
        x.update(kw)
        return _lib.Pool(*x.values())

    def pool_scales(**kw):
        x = dict(data=A, plane_stride=1 << 10, blocks=2)
        x.update(kw)
        return _lib.PoolScales(*x.values())

    def both(p, s):
        x = lib.fa_cache_update_8bit(p, s, A, A, A, A, 1 << 30, None)
        assert lib.fa_cache_compact_8bit(p, s, A, A, 1 << 30, None) == x
        return x

    assert both(pool(), None) == INVALID
    for kw in (dict(data=None), dict(blocks=0), dict(plane_stride=-1), dict(plane_stride=8)):
        assert both(pool(), pool_scales(**kw)) == INVALID, kw
    for kw in (dict(blocks=3), dict(blocks=8), dict(blocks=64)):
        assert both(pool(), pool_scales(**kw)) == UNSUPPORTED, kw
    assert both(pool(), pool_scales(data=A + 1)) == MISALIGNED
    assert both(pool(plane_stride=(1 << 20) + 8), pool_scales()) == INVALID
    assert both(pool(data=M), pool_scales()) == MISALIGNED


def test_wrappers_refuse_what_is_not_cuda():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        api.rotary(x, x, torch.zeros((8, 64)), torch.zeros(4, dtype=torch.int32))
    with pytest.raises(ValueError):
        api.cache_update(torch.zeros((2, 4, 2, 16, 64)).to(torch.float8_e4m3fn), torch.zeros((1, 4), dtype=torch.int32),
                         torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32), torch.zeros(1, dtype=torch.int32))
    for bad in ((0, 64), (10, 63), (10, 0)):
        with pytest.raises(ValueError):
            api.rotary_angles(*bad, device="cpu")


def test_angles_of_far_positions():
    """Formed in 64 bits: row 10^6 of the table is cos and sin of the exact angles to half a step of fp32 and the
    64-bit angle's own error (2^-53 of 10^6 twice, 2^-32)."""
    import math
    count, dim = 1000001, 32
    got = api.rotary_angles(count, dim, device="cpu")[-1].double()
    for j in range(dim // 2):
        x = (count - 1) * 10000.0 ** (-2 * j / dim)
        assert abs(float(got[j]) - math.cos(x)) <= 2.0 ** -25 + 2.0 ** -31
        assert abs(float(got[dim // 2 + j]) - math.sin(x)) <= 2.0 ** -25 + 2.0 ** -31


def test_least_power_of_the_plain_form():
    for most, scale, want in ((448.0, 1.0, 0), (448.0000305, 1.0, 1), (224.0, 1.0, -1), (1.0, 1.0, -8), (0.875, 1.0, -9),
                              (2.0 ** -140, 1.0, -148), (2.9e38, 2.0 ** -100, 219), (3.0, 0.3, -5)):
        assert least(most, scale) == want
        assert most <= 448 * scale * 2.0 ** want and most > 448 * scale * 2.0 ** (want - 1)
