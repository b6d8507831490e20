"""Binding of the paged key/value cache calls (include/kda.h): block tables and
slot maps from request lengths, the append of new keys and values, and the
attention of each request's new tokens over its cached keys.

As in ``kda.py``, argument marshalling only: outputs and the workspace are
allocated with torch, everything else runs in the library's CUDA kernels.
"""
from __future__ import annotations

import ctypes

import torch

from .kda import D, KDA_BF16, KDA_F32, KDAError, _check, _dtype_code, _p, _stream, load

KDA_E4M3 = 2
DEVERR_LENGTHS, DEVERR_NO_PAGES, DEVERR_PAGE = 8, 16, 32

_declared = False


def _lib():
    global _declared
    lib = load()
    if not _declared:
        P, I, L, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        lib.kda_paged_tables.argtypes = [P, P, I, L, P, I, P, I, P, P, I, I, P, P, P, P, P, P]
        lib.kda_paged_append.argtypes = [P, P, P, L, I, I, I, I, P, P, P, P, I, I, L, P, P]
        lib.kda_paged_attn.argtypes = [P, P, P, P, P, P, I, L, I, I, I, I, I, I, P, P, I, I, L, I, F, I, P, P, P, S, P, P]
        lib.kda_paged_attn_workspace_size.argtypes = [L, I, I, I]
        lib.kda_paged_attn_workspace_size.restype = S
        _declared = True
    return lib


def _on_device(*ts):
    """Every tensor contiguous and on one CUDA device (the caches are checked by
    _cache: their pages may lie apart)."""
    dev = None
    for t in ts:
        if t is None:
            continue
        if not t.is_cuda:
            raise KDAError("all tensors must be CUDA tensors")
        if not t.is_contiguous():
            raise KDAError("all tensors must be contiguous")
        if dev is None:
            dev = t.device
        elif t.device != dev:
            raise KDAError("all tensors must be on the same CUDA device")


def _typed(dtype, **ts):
    for name, t in ts.items():
        if t is not None and t.dtype != dtype:
            raise KDAError(f"{name} must be {str(dtype).replace('torch.', '')}")


def _cache_code(t) -> int:
    if t.dtype == torch.float8_e4m3fn:
        return KDA_E4M3
    return _dtype_code(t)


def _cache(x, k_cache, v_cache, k_scale, v_scale):
    """Geometry of the two caches, checked: (n_pages, Hkv, page_size, page stride)."""
    if k_cache.dim() != 4 or k_cache.shape[3] != D or k_cache.shape != v_cache.shape:
        raise KDAError("k_cache and v_cache must both be [pages, kv heads, page size, 128]")
    if k_cache.dtype != v_cache.dtype:
        raise KDAError("k_cache and v_cache must have the same dtype")
    n, h, ps, _ = k_cache.shape
    for t in (k_cache, v_cache):
        if not t.is_cuda or t.device != x.device:
            raise KDAError("the caches must be CUDA tensors on the inputs' device")
        if (n and h and ps) and t[0].is_contiguous() is False:
            raise KDAError("each page of a cache must be contiguous (pages may lie apart)")
    stride = k_cache.stride(0) if n > 1 else max(k_cache.stride(0), h * ps * D)
    if n > 1 and v_cache.stride(0) != stride:
        raise KDAError("k_cache and v_cache must have the same page stride")
    scales = (k_scale, v_scale)
    if (k_cache.dtype == torch.float8_e4m3fn) != all(s is not None for s in scales) or (k_scale is None) != (v_scale is None):
        raise KDAError("an e4m3 cache takes k_scale and v_scale, other caches none")
    for s in scales:
        if s is not None and (s.dtype != torch.float32 or tuple(s.shape) != (h,)):
            raise KDAError("k_scale and v_scale must be float32 [kv heads]")
    return n, h, ps, stride


def paged_tables(new_len, ctx_len, block_table, free_pages, free_head, T_total, page_size, n_pages, error_word=None):
    """kda_paged_tables: block_table [n, max_blocks] int32 gains the new pages in
    place.  new_len, ctx_len int32 [n]; free_pages int32 [n_free]; free_head int32 [1].
    Returns (slot_map int64 [T], positions int32 [T], cu_q int32 [n + 1], kv_len
    int32 [n], free_head_next int32 [1])."""
    lib = _lib()
    _on_device(new_len, ctx_len, block_table, free_pages, free_head, error_word)
    _typed(torch.int32, new_len=new_len, ctx_len=ctx_len, block_table=block_table, free_pages=free_pages,
           free_head=free_head, error_word=error_word)
    n = new_len.numel()
    if ctx_len.numel() != n or block_table.dim() != 2 or block_table.shape[0] != n or free_head.numel() != 1:
        raise KDAError("new_len and ctx_len must be [n], block_table [n, max_blocks], free_head [1]")
    dev = new_len.device
    T = int(T_total)
    slot_map = torch.empty(max(T, 0), dtype=torch.int64, device=dev)
    # one allocation for the int32 outputs; positions first (16-byte aligned)
    pad = (max(T, 0) + 3) // 4 * 4
    ints = torch.empty(pad + 2 * n + 2, dtype=torch.int32, device=dev)
    positions, cu_q, kv_len, head = ints[:max(T, 0)], ints[pad:pad + n + 1], ints[pad + n + 1:pad + 2 * n + 1], ints[pad + 2 * n + 1:]
    rc = lib.kda_paged_tables(_p(new_len), _p(ctx_len), n, T, _p(block_table), block_table.shape[1], _p(free_pages),
                              free_pages.numel(), _p(free_head), _p(head), int(page_size), int(n_pages), _p(slot_map),
                              _p(positions), _p(cu_q), _p(kv_len), _p(error_word), _stream(dev))
    _check(rc, "kda_paged_tables")
    return slot_map, positions, cu_q, kv_len, head


def paged_append(k, v, slot_map, k_cache, v_cache, k_scale=None, v_scale=None, error_word=None):
    """kda_paged_append: k, v [T, Hkv, 128] into the caches [pages, Hkv, page size,
    128] at slot_map int64 [T] (negative: skipped).  An e4m3 cache takes k_scale and
    v_scale float32 [Hkv]."""
    lib = _lib()
    _on_device(k, v, slot_map, k_scale, v_scale, error_word)
    _typed(torch.int64, slot_map=slot_map)
    _typed(torch.int32, error_word=error_word)
    n, h, ps, stride = _cache(k, k_cache, v_cache, k_scale, v_scale)
    if k.dim() != 3 or k.shape != v.shape or k.dtype != v.dtype or tuple(k.shape[1:]) != (h, D):
        raise KDAError("k and v must both be [T, kv heads, 128]")
    if slot_map.numel() != k.shape[0]:
        raise KDAError("slot_map must be [T]")
    rc = lib.kda_paged_append(_p(k), _p(v), _p(slot_map), k.shape[0], h, D, _dtype_code(k), _cache_code(k_cache),
                              _p(k_scale), _p(v_scale), _p(k_cache), _p(v_cache), n, ps, stride, _p(error_word),
                              _stream(k.device))
    _check(rc, "kda_paged_append")


def paged_attn_workspace_size(T_total: int, n_seqs: int, Hq: int, Hkv: int) -> int:
    return int(_lib().kda_paged_attn_workspace_size(T_total, n_seqs, Hq, Hkv))


def paged_attn(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q=0, sm_scale=D ** -0.5, window=0, k_scale=None,
               v_scale=None, out=None, lse=None, workspace=None, error_word=None):
    """kda_paged_attn: q [T, Hq, 128] over the caches [pages, Hkv, page size, 128]
    through block_table int32 [n, max_blocks]; cu_q int32 [n + 1] and kv_len int32 [n]
    as paged_tables gives them.  max_q: the most new tokens of one request (0: not
    known).  Returns (o in q's dtype, lse float32 [T, Hq])."""
    lib = _lib()
    _on_device(q, block_table, cu_q, kv_len, k_scale, v_scale, out, lse, workspace, error_word)
    _typed(torch.int32, block_table=block_table, cu_q=cu_q, kv_len=kv_len, error_word=error_word)
    _typed(torch.float32, lse=lse)
    n_pages, hkv, ps, stride = _cache(q, k_cache, v_cache, k_scale, v_scale)
    if q.dim() != 3 or q.shape[2] != D:
        raise KDAError("q must be [T, heads, 128]")
    T, hq, _ = q.shape
    n = kv_len.numel()
    if cu_q.numel() != n + 1 or block_table.dim() != 2 or block_table.shape[0] != n:
        raise KDAError("cu_q must be [n + 1], kv_len [n] and block_table [n, max_blocks]")
    o = out if out is not None else torch.empty_like(q)
    if o.shape != q.shape or o.dtype != q.dtype:
        raise KDAError("out must have q's shape and dtype")
    if lse is None:
        lse = torch.empty((T, hq), dtype=torch.float32, device=q.device)
    elif tuple(lse.shape) != (T, hq):
        raise KDAError("lse must be [T, heads]")
    if workspace is None:
        workspace = torch.empty(lib.kda_paged_attn_workspace_size(T, n, hq, hkv), dtype=torch.uint8, device=q.device)
    rc = lib.kda_paged_attn(_p(q), _p(k_cache), _p(v_cache), _p(block_table), _p(cu_q), _p(kv_len), n, T, int(max_q), hq,
                            hkv, D, _dtype_code(q), _cache_code(k_cache), _p(k_scale), _p(v_scale), n_pages, ps, stride,
                            block_table.shape[1], float(sm_scale), int(window), _p(o), _p(lse), _p(workspace),
                            workspace.numel() * workspace.element_size(), _p(error_word), _stream(q.device))
    _check(rc, "kda_paged_attn")
    return o, lse
