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

_DTYPES = {torch.bfloat16: 0, torch.float16: 1}  # fa_dtype


def _rows(name: str, t: torch.Tensor, like: Optional[torch.Tensor], heads: Optional[int] = None,
          tokens: Optional[int] = None) -> _lib.Rows:
    """fa_rows of a [T, H, d] tensor: d contiguous, the other strides positive multiples of 8."""
    if t.dim() != 3:
        raise ValueError(f"{name} must be [T, H, d], is {tuple(t.shape)}")
    T, H, d = t.shape
    if not t.is_cuda or t.dtype not in _DTYPES:
        raise ValueError(f"{name} must be a bfloat16 or float16 CUDA tensor")
    if like is not None and (t.dtype != like.dtype or t.device != like.device or d != like.shape[2]):
        raise ValueError(f"{name} must have q's (k's) dtype, device and head dim")
    if (heads is not None and H != heads) or (tokens is not None and T != tokens):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {(tokens, heads, d)}")
    st, sh, sd = t.stride()
    # the stride of a dimension of one element is never used: any valid value will do
    st, sh = (st if T > 1 else 8), (sh if H > 1 else 8)
    if (sd != 1 and d > 1) or st <= 0 or sh <= 0 or st % 8 or sh % 8:
        raise ValueError(f"{name} has strides {t.stride()}: the last must be 1, the others positive multiples of 8")
    return _lib.Rows(t.data_ptr(), st, sh)


def _int32(name: str, t: torch.Tensor, device, shape=None, dim: int = 1) -> torch.Tensor:
    if t.dtype != torch.int32 or t.dim() != dim or not t.is_contiguous() or t.device != device:
        raise ValueError(f"{name} must be a contiguous int32 tensor of {dim} dimension(s) on {device}")
    if shape is not None and tuple(t.shape) != shape:
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {shape}")
    return t


def _cu_of(cu: torch.Tensor, device) -> int:
    """The number of sequences of token offsets."""
    _int32("cu", cu, device)
    if cu.numel() < 1:
        raise ValueError("cu holds the offsets of B sequences and the end: at least one entry")
    return cu.numel() - 1


def _pages_of(k_cache: torch.Tensor, v_cache: torch.Tensor, table: torch.Tensor, like: torch.Tensor, hkv: int,
              B: int) -> _lib.Pages:
    """fa_pages of [n_pages, Hkv, page_size, d] caches and an int32 [>= B, width] table."""
    for name, c in (("k_cache", k_cache), ("v_cache", v_cache)):
        if c.dim() != 4 or c.dtype != like.dtype or c.device != like.device:
            raise ValueError(f"{name} must be [n_pages, Hkv, page_size, d] with k's dtype and device")
        if c.shape[0] < 1 or c.shape[1] != hkv or c.shape[3] != like.shape[2]:
            raise ValueError(f"{name} has shape {tuple(c.shape)}: {hkv} heads of {like.shape[2]} are expected")
    if k_cache.shape != v_cache.shape or k_cache.stride() != v_cache.stride():
        raise ValueError("k_cache and v_cache must have the same shape and strides")
    n, H, page, d = k_cache.shape
    sp, sh, st, sd = k_cache.stride()
    sp, sh = (sp if n > 1 else 8), (sh if H > 1 else 8)
    if sd != 1 or min(sp, sh, st) <= 0 or sp % 8 or sh % 8 or st % 8:
        raise ValueError(f"the cache has strides {k_cache.stride()}: the last must be 1, the others positive multiples of 8")
    if table.dtype != torch.int32 or table.dim() != 2 or table.device != like.device or table.shape[0] < B or table.shape[1] < 1:
        raise ValueError(f"table must be an int32 [slots, width] tensor on {like.device} with at least {B} rows")
    ts = table.stride(0) if table.shape[0] > 1 else table.shape[1]
    if (table.stride(1) != 1 and table.shape[1] > 1) or ts < table.shape[1]:
        raise ValueError("table must have contiguous rows that do not overlap")
    return _lib.Pages(k_cache.data_ptr(), v_cache.data_ptr(), sp, sh, st, n, page, table.data_ptr(), ts, table.shape[1])


def _serve(q, k, v, cu, scale, out, lse, workspace):
    """What forward_prompt and forward_tree share: the rows, the sizes and the outputs."""
    rq = _rows("q", q, None)
    T, Hq, d = q.shape
    rk, rv = _rows("k", k, q, tokens=T), _rows("v", v, q, heads=k.shape[1], tokens=T)
    Hkv = k.shape[1]
    if Hkv < 1 or Hq % Hkv:
        raise ValueError(f"{Hq} query heads do not share {Hkv} key/value heads evenly")
    B = _cu_of(cu, q.device)
    if out is None:
        out = torch.empty((T, Hq, d), dtype=q.dtype, device=q.device)
    ro = _rows("out", out, q, heads=Hq, tokens=T)
    if lse is None:
        lse = torch.empty((Hq, T), dtype=torch.float32, device=q.device)
    elif lse is False:
        lse = None
    elif lse.dtype != torch.float32 or tuple(lse.shape) != (Hq, T) or not lse.is_contiguous() or lse.device != q.device:
        raise ValueError("lse must be a contiguous float32 [Hq, T] tensor on q's device")
    if workspace is None:
        workspace = torch.empty(max(_tree_workspace(q.device.index, d), 1), dtype=torch.uint8, device=q.device)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != q.device:
        raise ValueError("workspace must be a contiguous uint8 tensor on q's device")
    scale = 1.0 / math.sqrt(d) if scale is None else float(scale)
    return rq, rk, rv, ro, out, lse, workspace, (B, T, Hq, Hkv, d, _DTYPES[q.dtype], scale)


_workspace_sizes = {}


def _tree_workspace(index: int, d: int) -> int:
    """fa_forward_tree_workspace_size on a device: the same for every call."""
    if (index, d) not in _workspace_sizes:
        with torch.cuda.device(index):
            _workspace_sizes[index, d] = int(_lib_fa().fa_forward_tree_workspace_size(d))
    return _workspace_sizes[index, d]


def forward_prompt(q, k, v, cu_seqlens, scale: Optional[float] = None, out=None, lse=None, workspace=None):
    """O, LSE of causal attention over whole prompts packed back to back (include/fa.h:
    fa_forward_prompt): q [T, Hq, d], k and v [T, Hkv, d] bfloat16 or float16, strided views of one
    projection welcome; cu_seqlens int32 [B + 1]; lse [Hq, T] (lse=False: none is written)."""
    rq, rk, rv, ro, out, lse, workspace, sizes = _serve(q, k, v, cu_seqlens, scale, out, lse, workspace)
    with torch.cuda.device(q.device):
        rc = _lib_fa().fa_forward_prompt(rq, rk, rv, ro, _p(lse), _p(cu_seqlens), *sizes, _p(workspace),
                                         workspace.numel(), _stream(q.device))
    _lib.check(rc, "fa_forward_prompt")
    return out, lse


def forward_tree(q, k, v, k_cache, v_cache, table, lens, cu_nodes, mask=None, scale: Optional[float] = None, out=None,
                 lse=None, workspace=None):
    """O, LSE of drafted tokens over a cache in pages and over each other (include/fa.h:
    fa_forward_tree): q [T, Hq, d], k and v [T, Hkv, d] of the drafted tokens, k_cache and v_cache
    [n_pages, Hkv, page_size, d], table int32 [slots, width], lens int32 [B] cached tokens, cu_nodes
    int32 [B + 1]. mask: int32 [T, words] from tree_mask, or None for a chain (one token a
    sequence is plain decoding). lse [Hq, T] (lse=False: none is written)."""
    rq, rk, rv, ro, out, lse, workspace, sizes = _serve(q, k, v, cu_nodes, scale, out, lse, workspace)
    pages = _pages_of(k_cache, v_cache, table, k, k.shape[1], sizes[0])
    _int32("lens", lens, q.device, (sizes[0],))
    words = 0
    if mask is not None:
        _int32("mask", mask, q.device, dim=2)
        words = mask.shape[1]
        if mask.shape[0] != q.shape[0] or words < 1:
            raise ValueError(f"mask has shape {tuple(mask.shape)}, expected ({q.shape[0]}, words >= 1)")
    with torch.cuda.device(q.device):
        rc = _lib_fa().fa_forward_tree(rq, rk, rv, ro, _p(lse), pages, _p(lens), _p(cu_nodes), _p(mask), words, *sizes,
                                       _p(workspace), workspace.numel(), _stream(q.device))
    _lib.check(rc, "fa_forward_tree")
    return out, lse


def tree_mask(parents, cu_nodes, words: int, out=None) -> torch.Tensor:
    """Which nodes each node of a tree sees, itself and its ancestors, as bits (include/fa.h:
    fa_tree_mask): parents int32 [T] (index within the sequence, negative for a root), cu_nodes int32
    [B + 1]; int32 [T, words], 32 nodes a word. One mask serves every layer."""
    if not parents.is_cuda:
        raise ValueError("parents must be a CUDA tensor")
    _int32("parents", parents, parents.device)
    B, T, words = _cu_of(cu_nodes, parents.device), parents.numel(), int(words)
    if words < 1:
        raise ValueError("words must be at least 1")
    if out is None:
        out = torch.empty((T, words), dtype=torch.int32, device=parents.device)
    _int32("out", out, parents.device, (T, words), dim=2)
    with torch.cuda.device(parents.device):
        rc = _lib_fa().fa_tree_mask(_p(parents), _p(cu_nodes), _p(out), words, B, T, _stream(parents.device))
    _lib.check(rc, "fa_tree_mask")
    return out


def cache_append(k, v, k_cache, v_cache, table, start, cu, rows=None) -> None:
    """Writes tokens into their pages (include/fa.h: fa_cache_append): token i of sequence b goes to
    position start[b] + i. k and v [Tkv, Hkv, d]; with rows (int32 [T]) token cu[b] + i is row
    rows[cu[b] + i] of them, else row cu[b] + i."""
    rk = _rows("k", k, None)
    T, Hkv, d = k.shape
    rv = _rows("v", v, k, heads=Hkv, tokens=T)
    B = _cu_of(cu, k.device)
    pages = _pages_of(k_cache, v_cache, table, k, Hkv, B)
    _int32("start", start, k.device, (B,))
    n = T
    if rows is not None:
        n = _int32("rows", rows, k.device).numel()
    with torch.cuda.device(k.device):
        rc = _lib_fa().fa_cache_append(rk, rv, pages, _p(start), _p(cu), _p(rows), B, n, T, Hkv, d, _stream(k.device))
    _lib.check(rc, "fa_cache_append")


def _pool_of(kv: torch.Tensor, table: torch.Tensor, lens: torch.Tensor, workspace):
    if not kv.is_cuda or kv.dtype not in _DTYPES or kv.dim() != 5 or kv.numel() == 0:
        raise ValueError("kv must be a bfloat16 or float16 CUDA tensor [planes, n_pages, Hkv, page_size, d]")
    if not kv[0].is_contiguous() or (kv.shape[0] > 1 and kv.stride(0) < kv[0].numel()):
        raise ValueError("each plane of kv must be contiguous, and apart from the others")
    _int32("table", table, kv.device, dim=2)
    if table.numel() == 0:
        raise ValueError("table must have at least one slot and one column")
    _int32("lens", lens, kv.device, (table.shape[0],))
    x, n, H, page, d = kv.shape
    pool = _lib.Pool(kv.data_ptr(), kv.stride(0) if x > 1 else 0, x, n, H, page, d, table.data_ptr(), lens.data_ptr(),
                     table.shape[0], table.shape[1])
    if workspace is None:
        need = int(_lib_fa().fa_cache_workspace_size(n, *table.shape))
        workspace = torch.empty(max(need, 1), dtype=torch.uint8, device=kv.device)
    elif workspace.dtype != torch.uint8 or not workspace.is_contiguous() or workspace.device != kv.device:
        raise ValueError("workspace must be a contiguous uint8 tensor on kv's device")
    return pool, workspace


def cache_update(kv, table, lens, src, new_lens, workspace=None) -> torch.Tensor:
    """Every slot s becomes the first min(new_lens[s], lens[src[s]]) tokens of slot src[s], with pages
    for new_lens[s] tokens (include/fa.h: fa_cache_update): forks, reorders, trims, frees and grows.
    kv [planes, n_pages, Hkv, page_size, d] holds K and V of every layer; table int32 [slots, width] and
    lens int32 [slots] are updated in place. Returns info, int32 [2]: the pages needed and the pages
    free (where more are needed than free, nothing has changed; -1, -1: invalid tables)."""
    pool, workspace = _pool_of(kv, table, lens, workspace)
    for name, t in (("src", src), ("new_lens", new_lens)):
        _int32(name, t, kv.device, (table.shape[0],))
    info = torch.empty(2, dtype=torch.int32, device=kv.device)
    with torch.cuda.device(kv.device):
        rc = _lib_fa().fa_cache_update(pool, _p(src), _p(new_lens), _p(info), _p(workspace), workspace.numel(),
                                       _stream(kv.device))
    _lib.check(rc, "fa_cache_update")
    return info


def cache_compact(kv, table, lens, workspace=None) -> torch.Tensor:
    """Moves the pages in use to the lowest ids, in every plane, and the table with them (include/fa.h:
    fa_cache_compact). Returns info, int32 [2]: the pages in use and the pages moved."""
    pool, workspace = _pool_of(kv, table, lens, workspace)
    info = torch.empty(2, dtype=torch.int32, device=kv.device)
    with torch.cuda.device(kv.device):
        rc = _lib_fa().fa_cache_compact(pool, _p(info), _p(workspace), workspace.numel(), _stream(kv.device))
    _lib.check(rc, "fa_cache_compact")
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
