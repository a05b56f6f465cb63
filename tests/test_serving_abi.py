"""The serving entry points reject bad arguments on the host, before any CUDA call (no GPU needed)."""

import ctypes

import pytest
import torch

from io_aware_exact_04_gb300 import _lib, api

OK, INVALID, UNSUPPORTED, MISALIGNED = 0, 1, 2, 3
A, M = 0x10000, 0x10008  # 16-byte aligned and misaligned fake addresses: never dereferenced


@pytest.fixture(scope="module")
def lib(built):
    return _lib.load("libfa.so")


def rows(data=A, st=1024, sh=64):
    return _lib.Rows(data, st, sh)


def pages(**kw):
    x = dict(k=A, v=A, page_stride=4096, head_stride=1024, token_stride=64, n_pages=8, page_size=16, table=A,
             table_stride=4, table_width=4)
    x.update(kw)
    return _lib.Pages(*x.values())


def prompt(lib, q=None, k=None, v=None, o=None, lse=A, cu=A, B=1, T=4, Hq=4, Hkv=2, d=64, dtype=0, scale=0.125):
    q, k, v, o = (rows() if x is None else x for x in (q, k, v, o))
    return lib.fa_forward_prompt(q, k, v, o, lse, cu, B, T, Hq, Hkv, d, dtype, scale, None)


def tree(lib, q=None, k=None, v=None, o=None, lse=A, cache=None, lens=A, cu=A, mask=None, words=0, B=1, T=4, Hq=4, Hkv=2,
         d=64, dtype=0, scale=0.125, ws=A, nbytes=1 << 40):
    q, k, v, o = (rows() if x is None else x for x in (q, k, v, o))
    cache = pages() if cache is None else cache
    return lib.fa_forward_tree(q, k, v, o, lse, cache, lens, cu, mask, words, B, T, Hq, Hkv, d, dtype, scale, ws, nbytes,
                               None)


@pytest.mark.parametrize("call", [prompt, tree])
def test_attention_argument_errors(lib, call):
    for d in (0, 32, 96, 256):
        assert call(lib, d=d) == UNSUPPORTED
    for kw in (dict(B=-1), dict(T=-1), dict(Hq=0), dict(Hkv=0), dict(Hq=5), dict(dtype=2), dict(dtype=-1), dict(scale=0.0),
               dict(scale=-1.0), dict(scale=float("inf")), dict(scale=float("nan")), dict(cu=None)):
        assert call(lib, **kw) == INVALID, kw
    for kw in (dict(Hq=129, Hkv=1), dict(Hq=131072, Hkv=65536), dict(B=(1 << 20) + 1), dict(T=(1 << 30) + 1)):
        assert call(lib, **kw) == UNSUPPORTED, kw
    for name in ("q", "k", "v", "o"):
        assert call(lib, **{name: rows(data=None)}) == INVALID
        assert call(lib, **{name: rows(data=M)}) == MISALIGNED
        for bad in (dict(st=0), dict(st=-64), dict(st=12), dict(sh=0), dict(sh=-8), dict(sh=63)):
            assert call(lib, **{name: rows(**bad)}) == INVALID, bad
        assert call(lib, **{name: rows(st=1 << 39)}) == UNSUPPORTED
    assert call(lib, lse=M) == MISALIGNED
    # nothing to do: pointers unused
    nothing = rows(data=None)
    assert call(lib, q=nothing, k=nothing, v=nothing, o=nothing, lse=None, cu=None, T=0) == OK
    assert call(lib, q=nothing, k=nothing, v=nothing, o=nothing, lse=None, cu=None, B=0) == OK


def test_tree_argument_errors(lib):
    for kw in (dict(k=None), dict(v=None), dict(table=None), dict(n_pages=0), dict(table_width=0), dict(table_stride=3),
               dict(page_stride=0), dict(head_stride=-8), dict(token_stride=60)):
        assert tree(lib, cache=pages(**kw)) == INVALID, kw
    for kw in (dict(page_size=8), dict(page_size=48), dict(page_size=512), dict(page_size=0),
               dict(table_width=1 << 27, table_stride=1 << 27)):
        assert tree(lib, cache=pages(**kw)) == UNSUPPORTED, kw
    assert tree(lib, cache=pages(k=M)) == MISALIGNED
    assert tree(lib, cache=pages(v=M)) == MISALIGNED
    assert tree(lib, lens=None) == INVALID
    assert tree(lib, ws=None) == INVALID
    assert tree(lib, ws=A + 16) == MISALIGNED
    assert tree(lib, mask=A, words=0) == INVALID
    assert tree(lib, mask=A, words=(1 << 20) + 1) == UNSUPPORTED
    assert lib.fa_forward_tree_workspace_size(96) == 0


def test_mask_argument_errors(lib):
    def call(parents=A, cu=A, mask=A, words=1, B=1, T=4):
        return lib.fa_tree_mask(parents, cu, mask, words, B, T, None)
    for kw in (dict(parents=None), dict(cu=None), dict(mask=None), dict(words=0), dict(B=-1), dict(T=-1)):
        assert call(**kw) == INVALID, kw
    assert call(words=(1 << 20) + 1) == UNSUPPORTED
    assert call(parents=None, cu=None, mask=None, T=0) == OK


def test_append_argument_errors(lib):
    def call(k=None, v=None, cache=None, start=A, cu=A, picked=None, B=1, T=4, Tkv=4, H=2, d=64):
        return lib.fa_cache_append(rows() if k is None else k, rows() if v is None else v, pages() if cache is None else cache,
                                   start, cu, picked, B, T, Tkv, H, d, None)
    for kw in (dict(k=rows(data=None)), dict(v=rows(data=None)), dict(k=rows(st=4)), dict(v=rows(sh=-64)), dict(start=None),
               dict(cu=None), dict(B=-1), dict(T=-1), dict(Tkv=-1), dict(H=0), dict(T=5), dict(picked=A, Tkv=0),
               dict(cache=pages(token_stride=4)), dict(cache=pages(k=None)), dict(cache=pages(n_pages=0))):
        assert call(**kw) == INVALID, kw
    for kw in (dict(d=80), dict(cache=pages(page_size=24)), dict(H=65536)):
        assert call(**kw) == UNSUPPORTED, kw
    for kw in (dict(k=rows(data=M)), dict(v=rows(data=M)), dict(cache=pages(v=M))):
        assert call(**kw) == MISALIGNED, kw
    assert call(start=None, cu=None, T=0, Tkv=0) == OK


def test_pool_argument_errors(lib):
    names = ("data", "plane_stride", "planes", "n_pages", "Hkv", "page_size", "d", "table", "lens", "slots", "table_width")

    def pool(**kw):
        x = dict(zip(names, (A, 8 * 2 * 16 * 64, 2, 8, 2, 16, 64, A, A, 3, 4)))
        x.update(kw)
        return _lib.Pool(*x.values())

    def update(p, src=A, new=A, info=A, ws=A, nbytes=1 << 40):
        return lib.fa_cache_update(p, src, new, info, ws, nbytes, None)

    def compact(p, info=A, ws=A, nbytes=1 << 40):
        return lib.fa_cache_compact(p, info, ws, nbytes, None)

    need = lib.fa_cache_workspace_size(8, 3, 4)
    assert need > 0
    for call in (update, compact):
        for kw in (dict(data=None), dict(table=None), dict(lens=None), dict(planes=0), dict(n_pages=0), dict(Hkv=0),
                   dict(slots=0), dict(table_width=0), dict(plane_stride=-8), dict(plane_stride=8 * 2 * 16 * 64 - 8),
                   dict(plane_stride=8 * 2 * 16 * 64 + 4)):
            assert call(pool(**kw)) == INVALID, kw
        for kw in (dict(page_size=20), dict(d=32), dict(n_pages=(1 << 28) + 1), dict(slots=(1 << 20) + 1),
                   dict(table_width=(1 << 26) + 1), dict(slots=1 << 20, table_width=1 << 10)):
            assert call(pool(**kw)) == UNSUPPORTED, kw
        assert call(pool(data=M)) == MISALIGNED
        assert call(pool(), ws=A + 64) == MISALIGNED
        assert call(pool(), info=None) == INVALID
        assert call(pool(), ws=None) == INVALID
        assert call(pool(), nbytes=need - 1) == INVALID
    for n, s, w in ((0, 3, 4), (8, 0, 4), (8, 3, 0), (-1, 3, 4), (8, 1 << 20, 1 << 10)):
        assert lib.fa_cache_workspace_size(n, s, w) == 0


def test_wrappers_refuse_host_tensors():
    x = torch.zeros((4, 2, 64), dtype=torch.bfloat16)
    i = torch.zeros(2, dtype=torch.int32)
    kv = torch.zeros((2, 4, 2, 16, 64), dtype=torch.bfloat16)
    t = torch.zeros((2, 4), dtype=torch.int32)
    for call in (lambda: api.forward_prompt(x, x, x, i), lambda: api.forward_tree(x, x, x, kv[0], kv[1], t, i[:1], i),
                 lambda: api.tree_mask(i, i, 1), lambda: api.cache_append(x, x, kv[0], kv[1], t, i[:1], i),
                 lambda: api.cache_update(kv, t, i, i, i), lambda: api.cache_compact(kv, t, i)):
        with pytest.raises(ValueError):
            call()
