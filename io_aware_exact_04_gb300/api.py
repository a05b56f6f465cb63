"""PyTorch-facing wrappers of the C ABI: argument checks and marshalling only.

PyTorch provides device memory and the current CUDA stream; every step of the
attention computation runs in the library's kernels.
"""

from __future__ import annotations

import ctypes
import math
from typing import Optional, Tuple

import torch

from . import _lib


def _lib_fa():
    return _lib.load("libfa.so")


def _p(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device: torch.device):
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _check_bhnd(name: str, t: torch.Tensor, shape=None):
    if not t.is_cuda:
        raise ValueError(f"{name} must be a CUDA tensor")
    if t.dtype != torch.bfloat16:
        raise ValueError(f"{name} must be bfloat16")
    if t.dim() != 4 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous [B, H, N, d] tensor")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _kv(kv_len: Optional[torch.Tensor], B: int, device) -> Optional[torch.Tensor]:
    if kv_len is None:
        return None
    if kv_len.dtype != torch.int32 or kv_len.shape != (B,) or not kv_len.is_contiguous():
        raise ValueError("kv_len must be a contiguous int32 tensor of shape [B]")
    if kv_len.device != device:
        raise ValueError("kv_len must live on the same device as q")
    return kv_len


def _kv_shape(q, k):
    """[B, H, N_k, d] of k: q's batch, heads and head dim with its own length."""
    _check_bhnd("k", k)
    if k.shape[0] != q.shape[0] or k.shape[1] != q.shape[1] or k.shape[3] != q.shape[3]:
        raise ValueError(f"k has shape {tuple(k.shape)}; q is {tuple(q.shape)} (only N may differ)")
    return tuple(k.shape)


def forward(q, k, v, causal: bool = False, scale: Optional[float] = None, kv_len=None, out=None,
            lse=None) -> Tuple[torch.Tensor, torch.Tensor]:
    """O, LSE of exact softmax attention (include/fa.h: fa_forward_qk). q is [B, H, N_q, d];
    k and v are [B, H, N_k, d] (N_k may differ; causal aligns the queries with the last keys)."""
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    kshape = _kv_shape(q, k)
    _check_bhnd("v", v, kshape)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q) if out is None else out
    _check_bhnd("out", o, q.shape)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if lse is None else lse
    kv = _kv(kv_len, B, q.device)
    with torch.cuda.device(q.device):
        rc = _lib_fa().fa_forward_qk(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, N, kshape[2], d, scale,
                                     int(bool(causal)), _p(kv), _stream(q.device))
    _lib.check(rc, "fa_forward_qk")
    return o, lse


def _check_hTd(name: str, t: torch.Tensor, shape=None):
    if not t.is_cuda or t.dtype != torch.bfloat16 or t.dim() != 3 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous bfloat16 CUDA tensor [H, T, d]")
    if shape is not None and tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")


def _cu(cu_seqlens: torch.Tensor, device) -> torch.Tensor:
    if cu_seqlens.dtype != torch.int32 or cu_seqlens.dim() != 1 or not cu_seqlens.is_contiguous():
        raise ValueError("cu_seqlens must be a contiguous int32 tensor [B + 1]")
    if cu_seqlens.device != device:
        raise ValueError("cu_seqlens must live on the same device as q")
    return cu_seqlens


def forward_varlen(q, k, v, cu_seqlens, max_seqlen: int, causal: bool = False, scale: Optional[float] = None):
    """O, LSE over packed sequences (include/fa.h: fa_forward_varlen): q, k, v [H, T, d], sequence
    b at rows cu_seqlens[b] .. cu_seqlens[b + 1]; lse [H, T]."""
    _check_hTd("q", q)
    H, T, d = q.shape
    _check_hTd("k", k, q.shape)
    _check_hTd("v", v, q.shape)
    cu = _cu(cu_seqlens, q.device)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    o = torch.empty_like(q)
    lse = torch.empty((H, T), dtype=torch.float32, device=q.device)
    with torch.cuda.device(q.device):
        rc = _lib_fa().fa_forward_varlen(_p(q), _p(k), _p(v), _p(o), _p(lse), _p(cu), cu.numel() - 1, H, T,
                                         int(max_seqlen), d, scale, int(bool(causal)), _stream(q.device))
    _lib.check(rc, "fa_forward_varlen")
    return o, lse


def backward_varlen(q, k, v, o, do, lse, cu_seqlens, max_seqlen: int, causal: bool = False,
                    scale: Optional[float] = None):
    """dQ, dK, dV over packed sequences (include/fa.h: fa_backward_varlen); shapes as forward_varlen."""
    _check_hTd("q", q)
    H, T, d = q.shape
    for name, t in (("k", k), ("v", v), ("o", o), ("do", do)):
        _check_hTd(name, t, q.shape)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (H, T) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [H, T] tensor")
    cu = _cu(cu_seqlens, q.device)
    B = cu.numel() - 1
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq, dk, dv = torch.empty_like(q), torch.empty_like(q), torch.empty_like(q)
    lib = _lib_fa()
    need = int(lib.fa_backward_varlen_workspace_size(B, H, T, d))
    work = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    with torch.cuda.device(q.device):
        rc = lib.fa_backward_varlen(_p(q), _p(k), _p(v), _p(o), _p(do), _p(lse), _p(dq), _p(dk), _p(dv), _p(cu), B, H,
                                    T, int(max_seqlen), d, scale, int(bool(causal)), _p(work), work.numel(),
                                    _stream(q.device))
    _lib.check(rc, "fa_backward_varlen")
    return dq, dk, dv


def forward_split(q, k, v, causal: bool = False, scale: Optional[float] = None, kv_len=None,
                  n_split: Optional[int] = None, with_lse: bool = False, out=None, workspace=None):
    """Inference forward with split keys (include/fa.h: fa_forward_split): O, and LSE when
    with_lse (else None). n_split defaults to the library's choice for the shape."""
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    kshape = _kv_shape(q, k)
    _check_bhnd("v", v, kshape)
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    lib = _lib_fa()
    if n_split is None:
        with torch.cuda.device(q.device):
            n_split = int(lib.fa_forward_split_count(B, H, N, kshape[2], d))
    o = torch.empty_like(q) if out is None else out
    _check_bhnd("out", o, q.shape)
    lse = torch.empty((B, H, N), dtype=torch.float32, device=q.device) if with_lse else None
    need = int(lib.fa_forward_split_workspace_size(B, H, N, d, n_split))
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    kv = _kv(kv_len, B, q.device)
    with torch.cuda.device(q.device):
        rc = lib.fa_forward_split(_p(q), _p(k), _p(v), _p(o), _p(lse), B, H, N, kshape[2], d, scale,
                                  int(bool(causal)), _p(kv), int(n_split), _p(workspace), workspace.numel(),
                                  _stream(q.device))
    _lib.check(rc, "fa_forward_split")
    return o, lse


def workspace_bytes(B: int, H: int, N: int, d: int) -> int:
    return int(_lib_fa().fa_backward_workspace_size(B, H, N, d))


def backward(q, k, v, o, do, lse, causal: bool = False, scale: Optional[float] = None, kv_len=None,
             dq=None, dk=None, dv=None, workspace=None):
    """dQ, dK, dV by recomputation from Q, K, V, O, dO and LSE (fa_backward_qk); shapes as
    for forward."""
    _check_bhnd("q", q)
    B, H, N, d = q.shape
    kshape = _kv_shape(q, k)
    for name, t, shp in (("v", v, kshape), ("o", o, q.shape), ("do", do, q.shape)):
        _check_bhnd(name, t, shp)
    if lse.dtype != torch.float32 or tuple(lse.shape) != (B, H, N) or not lse.is_contiguous():
        raise ValueError("lse must be a contiguous float32 [B, H, N] tensor")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    dq = torch.empty_like(q) if dq is None else dq
    dk = torch.empty_like(k) if dk is None else dk
    dv = torch.empty_like(k) if dv is None else dv
    need = workspace_bytes(B, H, N, d)
    if workspace is None:
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=q.device)
    kv = _kv(kv_len, B, q.device)
    with torch.cuda.device(q.device):
        rc = _lib_fa().fa_backward_qk(_p(q), _p(k), _p(v), _p(o), _p(do), _p(lse), _p(dq), _p(dk), _p(dv),
                                      B, H, N, kshape[2], d, scale, int(bool(causal)), _p(kv), _p(workspace),
                                      workspace.numel(), _stream(q.device))
    _lib.check(rc, "fa_backward_qk")
    return dq, dk, dv


def device_status(device=None):
    """(code, [code, site, blockIdx.x, blockIdx.y]) of the device status word; clears it."""
    dev = torch.device("cuda", torch.cuda.current_device()) if device is None else torch.device(device)
    detail = (ctypes.c_int * 4)()
    with torch.cuda.device(dev):
        rc = _lib_fa().fa_get_last_device_status_detail(_stream(dev), detail)
    return rc, list(detail)


# ------------------------------------------------------------------ serving
# Prompts, drafted trees over a cache in pages, and the cache's own work (include/fa.h, "serving").
# Their smallest calls take a few microseconds on the GPU, so the checks here are written to cost
# little where nothing is wrong: one condition a tensor, the reasons worked out only after it fails.

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}  # fa_dtype
_raw_stream = torch._C._cuda_getCurrentRawStream if hasattr(torch._C, "_cuda_getCurrentRawStream") else (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_FP32, _INT32, _UINT8 = torch.float32, torch.int32, torch.uint8


def _call(name: str, index: int, *args) -> None:
    """One entry point on device `index` and its current stream."""
    fn = getattr(_lib_fa(), name)
    if torch.cuda.current_device() == index:
        rc = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            rc = fn(*args, _raw_stream(index))
    if rc:
        _lib.check(rc, name)


def _first(name: str, t: torch.Tensor, dim: int) -> int:
    """The device of the tensor that the others of a call go by, once its type is one that is served."""
    if not t.is_cuda or t.dtype not in _DTYPES or t.dim() != dim:
        raise ValueError(f"{name} must be a bfloat16 or float16 CUDA tensor of {dim} dimensions")
    return t.get_device()


def _rows(name: str, t: torch.Tensor, index: int, dtype, T: int, H: int, d: int) -> _lib.Rows:
    """fa_rows of a [T, H, d] tensor: d contiguous, the other strides positive multiples of 8."""
    if t.dtype is not dtype or t.get_device() != index or t.shape != (T, H, d):  # (a CPU tensor's device is -1)
        raise ValueError(f"{name} must be a {dtype} tensor {(T, H, d)} on cuda:{index}, is {t.dtype} {tuple(t.shape)} on {t.device}")
    st, sh, sd = t.stride()
    # the stride of a dimension of one element is never used: any valid value will do
    if T <= 1:
        st = 8
    if H <= 1:
        sh = 8
    if (sd != 1 and d > 1) or st <= 0 or sh <= 0 or (st | sh) & 7:
        raise ValueError(f"{name} has strides {t.stride()}: the last must be 1, the others positive multiples of 8")
    return _lib.Rows(t.data_ptr(), st, sh)


def _ints(name: str, t: torch.Tensor, index: int, shape) -> int:
    """The address of a contiguous int32 tensor of a given shape."""
    if t.dtype is not _INT32 or t.get_device() != index or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {tuple(shape)} on cuda:{index}, is {t.dtype} "
                         f"{tuple(t.shape)} on {t.device}")
    return t.data_ptr()


def _offsets(cu: torch.Tensor, index: int):
    """The address of token offsets and how many sequences they bound."""
    n = cu.numel()
    if n < 1:
        raise ValueError("cu holds the offsets of B sequences and the end: int32 [B + 1]")
    return _ints("cu", cu, index, (n,)), n - 1


def _workspace(workspace, need: int, index: int):
    if workspace is None:
        return torch.empty(need, dtype=_UINT8, device=index)
    if workspace.dtype is not _UINT8 or workspace.get_device() != index or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous uint8 tensor on cuda:{index}")
    return workspace


def _pages(k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor, index: int, dtype, H: int, d: int,
           B: int, unit: int = 8) -> _lib.Pages:
    """fa_pages of [n_pages, Hkv, page_size, d] caches, `unit` elements in 16 bytes, and an int32 [>= B, width] table."""
    shape, strides = k_cache.shape, k_cache.stride()
    if len(shape) != 4 or v_cache.shape != shape or v_cache.stride() != strides or shape[1] != H or shape[3] != d or shape[0] < 1:
        raise ValueError(f"k_cache and v_cache must be [n_pages, {H}, page_size, {d}] with the same shape and strides, are "
                         f"{tuple(shape)} {strides} and {tuple(v_cache.shape)} {v_cache.stride()}")
    if (k_cache.dtype is not dtype or v_cache.dtype is not dtype or k_cache.get_device() != index or
            v_cache.get_device() != index):
        raise ValueError(f"k_cache and v_cache must be {dtype} tensors on cuda:{index}")
    n, _, page, _ = shape
    sp, sh, st, sd = strides
    if n == 1:
        sp = unit
    if H == 1:
        sh = unit
    if sd != 1 or sp <= 0 or sh <= 0 or st <= 0 or (sp | sh | st) & (unit - 1):
        raise ValueError(f"the cache has strides {strides}: the last must be 1, the others positive multiples of {unit}")
    if table.dtype is not _INT32 or table.get_device() != index or table.dim() != 2:
        raise ValueError(f"table must be an int32 [slots, width] tensor on cuda:{index}")
    slots, width = table.shape
    ts, tw = table.stride()
    if slots <= 1:
        ts = width
    if slots < B or width < 1 or (tw != 1 and width > 1) or ts < width:
        raise ValueError(f"table must have contiguous rows that do not overlap, {B} of them at least: is {(slots, width)} "
                         f"with strides {table.stride()}")
    return _lib.Pages(k_cache.data_ptr(), v_cache.data_ptr(), sp, sh, st, n, page, table.data_ptr(), ts, width)


_E4M3 = torch.float8_e4m3fn


def _cache(k_cache, v_cache, k_scale, v_scale, table, index: int, dtype, H: int, d: int, B: int):
    """fa_pages of a cache in 16 bits and None, or of one in 8 bits and its fa_scales: k_scale and v_scale float32
    [n_pages, Hkv, blocks], a block being page_size / blocks tokens."""
    if k_cache.dtype is not _E4M3:
        if k_scale is not None or v_scale is not None:
            raise ValueError(f"k_scale and v_scale belong to a cache of {_E4M3}, this one is {k_cache.dtype}")
        return _pages(k_cache, v_cache, table, index, dtype, H, d, B), None
    if k_scale is None or v_scale is None:
        raise ValueError("a cache in 8 bits needs k_scale and v_scale")
    pages = _pages(k_cache, v_cache, table, index, _E4M3, H, d, B, 16)
    n, _, page, _ = k_cache.shape
    shape, strides = k_scale.shape, k_scale.stride()
    for name, t in (("k_scale", k_scale), ("v_scale", v_scale)):
        if t.dtype is not _FP32 or t.get_device() != index or t.shape != shape or len(shape) != 3 or shape[0] != n or shape[1] != H:
            raise ValueError(f"{name} must be a float32 tensor ({n}, {H}, blocks) on cuda:{index}, is {t.dtype} "
                             f"{tuple(t.shape)} on {t.device}")
    blocks = shape[2]
    sp, sh, sb = strides
    if blocks < 1 or page % blocks or page // blocks not in (16, 32, 64, 128, 256):
        raise ValueError(f"{blocks} blocks of a page of {page} tokens: a block has 16, 32, 64, 128 or 256 of them")
    if v_scale.stride() != strides or (sb != 1 and blocks > 1):
        raise ValueError(f"k_scale and v_scale must have the same strides, the last 1: {k_scale.stride()}, {v_scale.stride()}")
    if n == 1:
        sp = 1
    if H == 1:
        sh = 1
    if sp < 1 or sh < 1:
        raise ValueError(f"the scales have strides {k_scale.stride()}: they must be positive")
    return pages, _lib.Scales(k_scale.data_ptr(), v_scale.data_ptr(), sp, sh, page // blocks)


def _serve(q, k, v, cu, scale, out, lse):
    """What forward_prompt and forward_tree share: the rows, the sizes and the outputs."""
    index, dtype = _first("q", q, 3), q.dtype
    T, Hq, d = q.shape
    if k.dim() != 3:
        raise ValueError(f"k must be [T, Hkv, d], is {tuple(k.shape)}")
    Hkv = k.shape[1]
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads do not share {Hkv} key/value heads evenly")
    at, B = _offsets(cu, index)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=dtype, device=index)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=_FP32, device=index)
    elif lse is False:
        lse = None
    elif lse.dtype is not _FP32 or lse.get_device() != index or lse.shape != (Hq, T) or not lse.is_contiguous():
        raise ValueError(f"lse must be a contiguous float32 tensor {(Hq, T)} on cuda:{index}")
    rows = (_rows("q", q, index, dtype, T, Hq, d), _rows("k", k, index, dtype, T, Hkv, d),
            _rows("v", v, index, dtype, T, Hkv, d), _rows("out", out, index, dtype, T, Hq, d),
            None if lse is None else lse.data_ptr())
    sizes = (B, T, Hq, Hkv, d, _DTYPES[dtype], 1.0 / math.sqrt(d) if scale is None else float(scale))
    return index, rows, at, sizes, out, lse


_workspace_sizes = {}


def _tree_workspace(index: int, d: int, name: str = "fa_forward_tree") -> int:
    """The workspace size of an entry point on a device: the same for every call."""
    if (name, index, d) not in _workspace_sizes:
        with torch.cuda.device(index):
            _workspace_sizes[name, index, d] = max(int(getattr(_lib_fa(), name + "_workspace_size")(d)), 1)
    return _workspace_sizes[name, index, d]


def forward_prompt(q, k, v, cu_seqlens, scale: Optional[float] = None, out=None, lse=None):
    """O, LSE of causal attention over whole prompts packed back to back (include/fa.h:
    fa_forward_prompt): q [T, Hq, d], k and v [T, Hkv, d] bfloat16 or float16, strided views of one
    projection welcome; cu_seqlens int32 [B + 1]; lse [Hq, T] (lse=False: none is written)."""
    index, rows, at, sizes, out, lse = _serve(q, k, v, cu_seqlens, scale, out, lse)
    _call("fa_forward_prompt", index, *rows, at, *sizes)
    return out, lse


def forward_tree(q, k, v, k_cache, v_cache, table, lens, cu_nodes, mask=None, scale: Optional[float] = None, out=None,
                 lse=None, workspace=None, k_scale=None, v_scale=None):
    """O, LSE of drafted tokens over a cache in pages and over each other (include/fa.h:
    fa_forward_tree, fa_forward_tree_8bit): q [T, Hq, d], k and v [T, Hkv, d] of the drafted tokens,
    k_cache and v_cache [n_pages, Hkv, page_size, d] of the same type, or float8_e4m3fn with k_scale and
    v_scale float32 [n_pages, Hkv, blocks]; table int32 [slots, width], lens int32 [B] cached tokens,
    cu_nodes int32 [B + 1]. mask: int32 [T, words] from tree_mask, or None for a chain (one token a
    sequence is plain decoding). lse [Hq, T] (lse=False: none is written)."""
    index, rows, at, sizes, out, lse = _serve(q, k, v, cu_nodes, scale, out, lse)
    B, T, _, Hkv, d = sizes[:5]
    pages, scales = _cache(k_cache, v_cache, k_scale, v_scale, table, index, q.dtype, Hkv, d, B)
    bits, words = None, 0
    if mask is not None:
        if mask.dim() != 2 or mask.shape[1] < 1:
            raise ValueError(f"mask must be int32 [T, words], is {tuple(mask.shape)}")
        words = mask.shape[1]
        bits = _ints("mask", mask, index, (T, words))
    name, cache = ("fa_forward_tree", (pages,)) if scales is None else ("fa_forward_tree_8bit", (pages, scales))
    workspace = _workspace(workspace, _tree_workspace(index, d, name), index)
    _call(name, index, *rows, *cache, _ints("lens", lens, index, (B,)), at, bits, words, *sizes, workspace.data_ptr(),
          workspace.numel())
    return out, lse


def tree_mask(parents, cu_nodes, words: int, out=None) -> torch.Tensor:
    """Which nodes each node of a tree sees, itself and its ancestors, as bits (include/fa.h:
    fa_tree_mask): parents int32 [T] (index within the sequence, negative for a root), cu_nodes int32
    [B + 1]; int32 [T, words], 32 nodes a word. One mask serves every layer."""
    if not parents.is_cuda or parents.dim() != 1:
        raise ValueError("parents must be an int32 CUDA tensor [T]")
    index, T, words = parents.get_device(), parents.shape[0], int(words)
    at, B = _offsets(cu_nodes, index)
    if words < 1:
        raise ValueError("words must be at least 1")
    if out is None:
        out = torch.empty((T, words), dtype=_INT32, device=index)
    _call("fa_tree_mask", index, _ints("parents", parents, index, (T,)), at, _ints("out", out, index, (T, words)), words,
          B, T)
    return out


def cache_append(k, v, k_cache, v_cache, table, start, cu, rows=None, k_scale=None, v_scale=None) -> None:
    """Writes tokens into their pages (include/fa.h: fa_cache_append, fa_cache_append_8bit): token i of
    sequence b goes to position start[b] + i. k and v [Tkv, Hkv, d]; with rows (int32 [T]) token cu[b] + i
    is row rows[cu[b] + i] of them, else row cu[b] + i. A cache of float8_e4m3fn takes k_scale and v_scale,
    which are updated with it."""
    index, dtype = _first("k", k, 3), k.dtype
    Tkv, H, d = k.shape
    at, B = _offsets(cu, index)
    pages, scales = _cache(k_cache, v_cache, k_scale, v_scale, table, index, dtype, H, d, B)
    T, pick = Tkv, None
    if rows is not None:
        T = rows.shape[0] if rows.dim() == 1 else -1
        pick = _ints("rows", rows, index, (T,))
    given = (_rows("k", k, index, dtype, Tkv, H, d), _rows("v", v, index, dtype, Tkv, H, d), pages)
    where = (_ints("start", start, index, (B,)), at, pick, B, T, Tkv, H, d)
    if scales is None:
        _call("fa_cache_append", index, *given, *where)
    else:
        _call("fa_cache_append_8bit", index, *given, scales, *where, _DTYPES[dtype])


def rotary_angles(positions: int, dim: int, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """float32 [positions, dim]: the cosines of position i's angles i base^(-2 j / dim), j < dim / 2, then
    their sines, formed in 64 bits."""
    if dim < 2 or dim % 2 or positions < 1:
        raise ValueError(f"{positions} positions of {dim} elements: dim must be even, both positive")
    f = base ** (-torch.arange(0, dim, 2, dtype=torch.float64, device=device) / dim)
    x = torch.arange(positions, dtype=torch.float64, device=device)[:, None] * f
    return torch.cat([torch.cos(x), torch.sin(x)], 1).float()


def _angles(angles: torch.Tensor, positions, interleaved: bool, index: int, T: int) -> _lib.Rotary:
    if angles.dtype is not _FP32 or angles.get_device() != index or angles.dim() != 2 or angles.shape[0] < 1:
        raise ValueError(f"angles must be a float32 tensor [positions, dim] on cuda:{index}")
    count, dim = angles.shape
    st, se = angles.stride()
    if count == 1:
        st = dim
    if se != 1 or st < dim or st % 4 or dim < 16 or dim % 16:
        raise ValueError(f"angles {tuple(angles.shape)} with strides {angles.stride()}: dim must be a multiple of 16, rows "
                         f"contiguous, apart, a multiple of 4 between them")
    at = None if positions is None else _ints("positions", positions, index, (T,))
    return _lib.Rotary(angles.data_ptr(), st, count, dim, int(bool(interleaved)), at)


def _rotated(name: str, t, out, index: int, dtype, T: int, H: int, d: int):
    """fa_rows of a tensor to rotate and of its result (None: a new one)."""
    rows = _rows(name, t, index, dtype, T, H, d)
    if out is None:
        out = torch.empty((T, H, d), dtype=dtype, device=index)
        return rows, _lib.Rows(out.data_ptr(), H * d, d), out
    return rows, _rows(name + "_out", out, index, dtype, T, H, d), out


def rotary(q, k, angles, positions, interleaved: bool = False, q_out=None, k_out=None):
    """Queries [T, Hq, d] and keys [T, Hkv, d] rotated by the angles (rotary_angles) of their positions,
    int32 [T] (include/fa.h: fa_rotary_append without a cache): the nodes of a draft, say. Returns both;
    q_out=q, k_out=k rotates in place."""
    index, dtype = _first("q", q, 3), q.dtype
    T, Hq, d = q.shape
    if k.dim() != 3:
        raise ValueError(f"k must be [T, Hkv, d], is {tuple(k.shape)}")
    Hkv = k.shape[1]
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads do not share {Hkv} key/value heads evenly")
    if positions is None:
        raise ValueError("positions are needed without a cache")
    turn = _angles(angles, positions, interleaved, index, T)
    rq, ro, q_out = _rotated("q", q, q_out, index, dtype, T, Hq, d)
    rk, rko, k_out = _rotated("k", k, k_out, index, dtype, T, Hkv, d)
    _call("fa_rotary_append", index, rq, rk, None, ro, rko, None, None, turn, None, None, 0, T, Hq, Hkv, d, _DTYPES[dtype])
    return q_out, k_out


def rotary_append(q, k, v, k_cache, v_cache, table, start, cu, angles, positions=None, interleaved: bool = False, q_out=None,
                  k_out=None, k_scale=None, v_scale=None):
    """Rotates the queries [T, Hq, d] and keys [T, Hkv, d] of new tokens by the angles (rotary_angles) of their
    positions and writes the rotated keys and v [T, Hkv, d] into their pages, in one pass (include/fa.h:
    fa_rotary_append): token i of sequence b goes to position start[b] + i, which is its position for the
    angles too unless positions (int32 [T]) says another. Caches as for cache_append. Returns the rotated
    q and k, for forward_prompt or forward_tree; q_out=q, k_out=k rotates in place."""
    index, dtype = _first("q", q, 3), q.dtype
    T, Hq, d = q.shape
    if k.dim() != 3:
        raise ValueError(f"k must be [T, Hkv, d], is {tuple(k.shape)}")
    Hkv = k.shape[1]
    if Hkv < 1 or Hq < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads do not share {Hkv} key/value heads evenly")
    at, B = _offsets(cu, index)
    pages, scales = _cache(k_cache, v_cache, k_scale, v_scale, table, index, dtype, Hkv, d, B)
    turn = _angles(angles, positions, interleaved, index, T)
    rq, ro, q_out = _rotated("q", q, q_out, index, dtype, T, Hq, d)
    rk, rko, k_out = _rotated("k", k, k_out, index, dtype, T, Hkv, d)
    _call("fa_rotary_append", index, rq, rk, _rows("v", v, index, dtype, T, Hkv, d), ro, rko, pages, scales, turn,
          _ints("start", start, index, (B,)), at, B, T, Hq, Hkv, d, _DTYPES[dtype])
    return q_out, k_out


def _pool(kv: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, scales):
    if kv.dtype is not _E4M3:
        index, more = _first("kv", kv, 5), ()
        if scales is not None:
            raise ValueError(f"scales belong to a pool of {_E4M3}, this one is {kv.dtype}")
    elif kv.dim() != 5 or not kv.is_cuda:
        raise ValueError("kv must be a CUDA tensor of 5 dimensions")
    else:
        index, more = kv.get_device(), (_pool_scales(kv, scales),)
    x, n, H, page, d = kv.shape
    sx, sn, sh, st, sd = kv.stride()
    plane = n * H * page * d
    if plane == 0 or x == 0:
        raise ValueError("kv must have at least one plane, page, head and token")
    if x == 1:
        sx = 0
    if ((n > 1 and sn != H * page * d) or (H > 1 and sh != page * d) or (page > 1 and st != d) or (d > 1 and sd != 1) or
            (x > 1 and sx < plane)):
        raise ValueError(f"each plane of kv must be contiguous, and apart from the others: strides {kv.stride()}")
    if table.dim() != 2 or table.shape[0] < 1 or table.shape[1] < 1:
        raise ValueError("table must be int32 [slots, width] with at least one slot and one column")
    slots, width = table.shape
    pool = _lib.Pool(kv.data_ptr(), sx, x, n, H, page, d, _ints("table", table, index, (slots, width)),
                     _ints("lens", lens, index, (slots,)), slots, width)
    return index, slots, (pool, *more), (n, slots, width)


def _pool_scales(kv: torch.Tensor, scales) -> _lib.PoolScales:
    """fa_pool_scales of a pool of e4m3: float32 [planes, n_pages, Hkv, blocks], every plane contiguous."""
    x, n, H, page, _ = kv.shape
    if (scales is None or scales.dtype is not _FP32 or scales.device != kv.device or scales.dim() != 4 or
            scales.shape[:3] != (x, n, H) or scales.shape[3] < 1):
        raise ValueError(f"a pool in 8 bits needs scales, a float32 tensor {(x, n, H)} + (blocks,) on {kv.device}")
    blocks = scales.shape[3]
    sx, sn, sh, sb = scales.stride()
    if x == 1:
        sx = 0
    if (n > 1 and sn != H * blocks) or (H > 1 and sh != blocks) or (blocks > 1 and sb != 1) or (x > 1 and sx < n * H * blocks):
        raise ValueError(f"each plane of the scales must be contiguous, and apart from the others: strides {scales.stride()}")
    return _lib.PoolScales(scales.data_ptr(), sx, blocks)


def _pool_workspace(workspace, sizes, index: int):
    need = 1 if workspace is not None else max(int(_lib_fa().fa_cache_workspace_size(*sizes)), 1)
    return _workspace(workspace, need, index)


def cache_update(kv, table, lens, src, new_lens, workspace=None, scales=None) -> torch.Tensor:
    """Every slot s becomes the first min(new_lens[s], lens[src[s]]) tokens of slot src[s], with pages
    for new_lens[s] tokens (include/fa.h: fa_cache_update): forks, reorders, trims, frees and grows.
    kv [planes, n_pages, Hkv, page_size, d] holds K and V of every layer (float8_e4m3fn: with scales, float32
    [planes, n_pages, Hkv, blocks]); table int32 [slots, width] and lens int32 [slots] are updated in place.
    Returns info, int32 [2]: the pages needed and the pages free (where more are needed than free, nothing has
    changed; -1, -1: invalid tables)."""
    index, slots, pool, sizes = _pool(kv, table, lens, scales)
    workspace = _pool_workspace(workspace, sizes, index)
    info = torch.empty(2, dtype=_INT32, device=index)
    _call("fa_cache_update" if len(pool) == 1 else "fa_cache_update_8bit", index, *pool,
          _ints("src", src, index, (slots,)), _ints("new_lens", new_lens, index, (slots,)), info.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return info


def cache_compact(kv, table, lens, workspace=None, scales=None) -> torch.Tensor:
    """Moves the pages in use to the lowest ids, in every plane (with its scales, as for cache_update), and the
    table with them (include/fa.h: fa_cache_compact). Returns info, int32 [2]: the pages in use and the pages moved."""
    index, _, pool, sizes = _pool(kv, table, lens, scales)
    workspace = _pool_workspace(workspace, sizes, index)
    info = torch.empty(2, dtype=_INT32, device=index)
    _call("fa_cache_compact" if len(pool) == 1 else "fa_cache_compact_8bit", index, *pool, info.data_ptr(),
          workspace.data_ptr(), workspace.numel())
    return info


class _Attention(torch.autograd.Function):
    @staticmethod
    def forward(ctx, q, k, v, causal, scale, kv_len):
        o, lse = forward(q, k, v, causal=causal, scale=scale, kv_len=kv_len)
        ctx.save_for_backward(q, k, v, o, lse, kv_len if kv_len is not None else torch.empty(0))
        ctx.causal, ctx.scale, ctx.has_kv = causal, scale, kv_len is not None
        return o

    @staticmethod
    def backward(ctx, do):
        q, k, v, o, lse, kv = ctx.saved_tensors
        dq, dk, dv = backward(q, k, v, o, do.contiguous(), lse, causal=ctx.causal, scale=ctx.scale,
                              kv_len=kv if ctx.has_kv else None)
        return dq, dk, dv, None, None, None


def attention(q, k, v, causal: bool = False, scale: Optional[float] = None, kv_len=None) -> torch.Tensor:
    """Differentiable exact attention: O only; only the LSE is kept for backward."""
    return _Attention.apply(q, k, v, causal, scale, kv_len)
