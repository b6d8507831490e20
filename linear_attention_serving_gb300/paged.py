"""Binding of the paged key/value cache calls (include/kda.h): block tables and
slot maps from request lengths, the append of new keys and values, and the
attention of each request's new tokens over its cached keys.

As in ``kda.py``, argument marshalling only: outputs and the workspace are
allocated with torch, everything else runs in the library's CUDA kernels.  The
smallest calls take a few microseconds on the GPU, so a call first goes through
``_paged_fast`` (csrc_py/paged_fast.cpp), which makes the same checks and the same
call of the library in compiled code.  What it does not take, it leaves undone
and answers None; the checks here then say what is wrong, or make the call.  Where
it cannot be built or loaded (a warning says so), all calls are made here.
"""
from __future__ import annotations

import ctypes
import importlib.util
import warnings

import torch

from . import _build
from .kda import D, KDA_BF16, KDA_F32, KDAError, _check, load

KDA_E4M3 = 2
DEVERR_LENGTHS, DEVERR_NO_PAGES, DEVERR_PAGE = 8, 16, 32

_I32, _I64, _F32, _E4M3 = torch.int32, torch.int64, torch.float32, torch.float8_e4m3fn
_CODE = {torch.bfloat16: KDA_BF16, torch.float32: KDA_F32}
_CACHE_CODE = {**_CODE, _E4M3: KDA_E4M3}
_declared = None


def _not_loaded(*args):
    """Stands where the compiled calls will be until the first call loads them."""
    _lib()


_fast_tables = _fast_append = _fast_attn = _fast_rope = _fast_rope_append = _fast_verify = _not_loaded


def _load_fast(lib):
    global _fast_tables, _fast_append, _fast_attn, _fast_rope, _fast_rope_append, _fast_verify
    spec = importlib.util.spec_from_file_location("_paged_fast", _build.build_fast())
    fast = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(fast)
    fast.init(*(ctypes.cast(f, ctypes.c_void_p).value for f in (
        lib.kda_paged_tables, lib.kda_paged_append, lib.kda_paged_attn_sinks, lib.kda_paged_attn_workspace_size,
        lib.kda_qk_rope, lib.kda_paged_rope_append, lib.kda_verify_drafts, lib.kda_verify_drafts_workspace_size)))
    _fast_tables, _fast_append, _fast_attn = fast.tables, fast.append, fast.attn
    _fast_rope, _fast_rope_append, _fast_verify = fast.rope, fast.rope_append, fast.verify


def _lib():
    global _declared
    if _declared is None:
        lib = load()
        P, I, L, F, S = ctypes.c_void_p, ctypes.c_int, ctypes.c_int64, ctypes.c_float, ctypes.c_size_t
        G = ctypes.c_double
        lib.kda_paged_tables.argtypes = [P, P, I, L, P, I, P, I, P, P, I, I, P, P, P, P, P, P]
        lib.kda_paged_append.argtypes = [P, P, P, L, I, I, I, I, P, P, P, P, I, I, L, P, P]
        lib.kda_paged_attn.argtypes = [P, P, P, P, P, P, I, L, I, I, I, I, I, I, P, P, I, I, L, I, F, I, P, P, P, S, P, P]
        lib.kda_paged_attn_sinks.argtypes = [P, P, P, P, P, P, I, L, I, I, I, I, I, I, P, P, I, I, L, I, F, I, I, P, P, P, S, P, P]
        lib.kda_rope_frequencies.argtypes = [I, G, I, G, G, G, G, P, P]
        lib.kda_qk_rope.argtypes = [P, P, P, P, F, P, P, F, L, I, I, I, I, I, I, L, L, P, P, L, L, P]
        lib.kda_paged_rope_append.argtypes = [P, P, P, P, P, P, F, P, P, F, L, I, I, I, I, I, I, I, L, L, L, P, L, P, P, P, P, I,
                                              I, L, P, P]
        lib.kda_verify_drafts.argtypes = [P, P, P, P, P, I, I, I, I, L, L, L, L, P, P, P, S, P, P]
        lib.kda_verify_drafts_workspace_size.argtypes = [I, I, I, I]
        lib.kda_verify_drafts_workspace_size.restype = S
        lib.kda_paged_attn_workspace_size.argtypes = [L, I, I, I]
        lib.kda_paged_attn_workspace_size.restype = S
        try:
            _load_fast(lib)
        except Exception as e:  # no host compiler or headers, a directory that cannot be written
            warnings.warn(f"paged calls take the plain binding, 4 to 20 us a call slower on the host: {e}", RuntimeWarning)
        _declared = lib
    return _declared


try:  # the stream's address without a Stream object around it
    _raw_stream = torch._C._cuda_getCurrentRawStream
except AttributeError:
    def _raw_stream(index):
        return torch.cuda.current_stream(index).cuda_stream


def _on_device(*ts):
    """Every tensor contiguous and on one CUDA device; returns its index.  (The
    caches are checked by _cache: their pages may lie apart.)"""
    index = ts[0].get_device()
    for t in ts:
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            index = -1
    if index < 0:
        given = [t for t in ts if t is not None]
        if not all(t.is_cuda for t in given):
            raise KDAError("all tensors must be CUDA tensors")
        if not all(t.is_contiguous() for t in given):
            raise KDAError("all tensors must be contiguous")
        raise KDAError("all tensors must be on the same CUDA device")
    return index


def _typed(dtype, names, *ts):
    for name, t in zip(names.split(), ts):
        if t is not None and t.dtype is not dtype:
            raise KDAError(f"{name} must be {str(dtype).replace('torch.', '')}")


def _fit(x, bits=32):
    return -2 ** (bits - 1) <= x < 2 ** (bits - 1)


def _ints(names, *xs):
    """What the library takes as 32 bits fits them (ctypes would cut it down to them)."""
    for name, x in zip(names.split(), xs):
        if not _fit(x):
            raise KDAError(f"{name} must fit 32 bits")


def _p(t):
    return None if t is None else t.data_ptr()


def _cache(index, k_cache, v_cache, k_scale, v_scale):
    """Geometry of the two caches, checked: (n_pages, Hkv, page_size, page stride, type)."""
    shape = k_cache.shape
    if len(shape) != 4 or shape[3] != D or shape != v_cache.shape:
        raise KDAError("k_cache and v_cache must both be [pages, kv heads, page size, 128]")
    dtype = k_cache.dtype
    if dtype is not v_cache.dtype:
        raise KDAError("k_cache and v_cache must have the same dtype")
    if dtype not in _CACHE_CODE:
        raise KDAError(f"unsupported cache dtype {dtype}: bfloat16, float32 or float8_e4m3fn")
    if k_cache.get_device() != index or v_cache.get_device() != index:
        raise KDAError("the caches must be CUDA tensors on the inputs' device")
    n, h, ps, _ = shape
    if k_cache.is_contiguous() and v_cache.is_contiguous():
        stride = h * ps * D
    else:
        a, b = k_cache.stride(), v_cache.stride()
        if a[1:] != (ps * D, D, 1) or b[1:] != a[1:]:
            raise KDAError("each page of a cache must be contiguous (pages may lie apart)")
        if n > 1 and a[0] != b[0]:
            raise KDAError("k_cache and v_cache must have the same page stride")
        stride = a[0] if n > 1 else max(a[0], h * ps * D)
    if dtype is _E4M3:
        if k_scale is None or v_scale is None:
            raise KDAError("an e4m3 cache takes k_scale and v_scale")
        _typed(_F32, "k_scale v_scale", k_scale, v_scale)
        if k_scale.numel() != h or v_scale.numel() != h:
            raise KDAError("k_scale and v_scale must be [kv heads]")
    elif k_scale is not None or v_scale is not None:
        raise KDAError("k_scale and v_scale belong to an e4m3 cache")
    return n, h, ps, stride, _CACHE_CODE[dtype]


def paged_tables(new_len, ctx_len, block_table, free_pages, free_head, T_total, page_size, n_pages, error_word=None):
    """kda_paged_tables: block_table [n, max_blocks] int32 gains the new pages in
    place.  new_len, ctx_len int32 [n]; free_pages int32 [n_free]; free_head int32 [1].
    Returns (slot_map int64 [T], positions int32 [T], cu_q int32 [n + 1], kv_len
    int32 [n], free_head_next int32 [1])."""
    done = _fast_tables(new_len, ctx_len, block_table, free_pages, free_head, T_total, page_size, n_pages, error_word)
    if done is not None:
        return done
    lib = _declared or _lib()
    index = _on_device(new_len, ctx_len, block_table, free_pages, free_head, error_word)
    _typed(_I32, "new_len ctx_len block_table free_pages free_head error_word", new_len, ctx_len, block_table, free_pages,
           free_head, error_word)
    n = new_len.numel()
    if ctx_len.numel() != n or block_table.dim() != 2 or block_table.shape[0] != n or free_head.numel() != 1:
        raise KDAError("new_len and ctx_len must be [n], block_table [n, max_blocks], free_head [1]")
    T = int(T_total)
    if T < 0:
        raise KDAError("T_total must not be negative")
    _ints("n max_blocks n_free page_size n_pages", n, block_table.shape[1], free_pages.numel(), page_size, n_pages)
    slot_map = new_len.new_empty(T, dtype=_I64)
    positions, cu_q, kv_len, head = new_len.new_empty(T + 2 * n + 2).split_with_sizes((T, n + 1, n, 1))
    with torch.cuda.device(index):  # (the library launches on the current device)
        rc = lib.kda_paged_tables(new_len.data_ptr(), ctx_len.data_ptr(), n, T, block_table.data_ptr(), block_table.shape[1],
                                  free_pages.data_ptr(), free_pages.numel(), free_head.data_ptr(), head.data_ptr(),
                                  page_size, n_pages, slot_map.data_ptr(), positions.data_ptr(), cu_q.data_ptr(),
                                  kv_len.data_ptr(), _p(error_word), _raw_stream(index))
    if rc:
        _check(rc, "kda_paged_tables")
    return slot_map, positions, cu_q, kv_len, head


def paged_append(k, v, slot_map, k_cache, v_cache, k_scale=None, v_scale=None, error_word=None):
    """kda_paged_append: k, v [T, Hkv, 128] into the caches [pages, Hkv, page size,
    128] at slot_map int64 [T] (negative: skipped).  An e4m3 cache takes k_scale and
    v_scale float32 [Hkv]."""
    if _fast_append(k, v, slot_map, k_cache, v_cache, k_scale, v_scale, error_word) is not None:
        return
    lib = _declared or _lib()
    index = _on_device(k, v, slot_map, k_scale, v_scale, error_word)
    n, h, ps, stride, code = _cache(index, k_cache, v_cache, k_scale, v_scale)
    _typed(_I64, "slot_map", slot_map)
    _typed(_I32, "error_word", error_word)
    shape = k.shape
    if len(shape) != 3 or shape[1] != h or shape[2] != D or v.shape != shape or k.dtype is not v.dtype:
        raise KDAError("k and v must both be [T, kv heads, 128], of one dtype")
    if k.dtype not in _CODE:
        raise KDAError(f"unsupported dtype {k.dtype}: k and v must be bfloat16 or float32")
    T = shape[0]
    if slot_map.numel() != T:
        raise KDAError("slot_map must be [T]")
    with torch.cuda.device(index):
        rc = lib.kda_paged_append(k.data_ptr(), v.data_ptr(), slot_map.data_ptr(), T, h, D, _CODE[k.dtype], code, _p(k_scale),
                                  _p(v_scale), k_cache.data_ptr(), v_cache.data_ptr(), n, ps, stride, _p(error_word),
                                  _raw_stream(index))
    if rc:
        _check(rc, "kda_paged_append")


def paged_attn_workspace_size(T_total: int, n_seqs: int, Hq: int, Hkv: int) -> int:
    """Bytes of workspace that paged_attn needs (0 for shapes it does not take)."""
    if not (_fit(T_total, 64) and _fit(n_seqs) and _fit(Hq) and _fit(Hkv)):
        return 0
    return int(_lib().kda_paged_attn_workspace_size(T_total, n_seqs, Hq, Hkv))


def paged_attn(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q=0, sm_scale=D ** -0.5, window=0, k_scale=None,
               v_scale=None, out=None, lse=None, workspace=None, error_word=None, sinks=0):
    """kda_paged_attn: q [T, Hq, 128] over the caches [pages, Hkv, page size, 128]
    through block_table int32 [n, max_blocks]; cu_q int32 [n + 1] and kv_len int32 [n]
    as paged_tables gives them.  max_q: the most new tokens of one request (0: not
    known).  sinks: the first tokens of each request, which a window leaves visible.
    Returns (o in q's dtype, lse float32 [T, Hq])."""
    done = _fast_attn(q, k_cache, v_cache, block_table, cu_q, kv_len, max_q, sm_scale, window, k_scale, v_scale, out, lse,
                      workspace, error_word, sinks)
    if done is not None:
        return done
    lib = _declared or _lib()
    index = _on_device(q, block_table, cu_q, kv_len, k_scale, v_scale, out, lse, workspace, error_word)
    n_pages, hkv, ps, stride, code = _cache(index, k_cache, v_cache, k_scale, v_scale)
    _typed(_I32, "block_table cu_q kv_len error_word", block_table, cu_q, kv_len, error_word)
    shape, dtype = q.shape, q.dtype
    if len(shape) != 3 or shape[2] != D:
        raise KDAError("q must be [T, heads, 128]")
    if dtype not in _CODE:
        raise KDAError(f"unsupported dtype {dtype}: q must be bfloat16 or float32")
    T, hq, _ = shape
    n = kv_len.numel()
    if cu_q.numel() != n + 1 or block_table.dim() != 2 or block_table.shape[0] != n:
        raise KDAError("cu_q must be [n + 1], kv_len [n] and block_table [n, max_blocks]")
    _ints("n heads max_blocks max_q window sinks", n, hq, block_table.shape[1], max_q, window, sinks)
    if out is None:
        out = torch.empty_like(q)
    elif out.shape != shape or out.dtype is not dtype:
        raise KDAError("out must have q's shape and dtype")
    if lse is None:
        lse = q.new_empty(T, hq, dtype=_F32)
    elif lse.shape != shape[:2] or lse.dtype is not _F32:
        raise KDAError("lse must be float32 [T, heads]")
    if workspace is None:
        workspace = q.new_empty(lib.kda_paged_attn_workspace_size(T, n, hq, hkv), dtype=torch.uint8)
    with torch.cuda.device(index):
        call, beside = (lib.kda_paged_attn_sinks, (sinks,)) if sinks else (lib.kda_paged_attn, ())
        rc = call(q.data_ptr(), k_cache.data_ptr(), v_cache.data_ptr(), block_table.data_ptr(), cu_q.data_ptr(), kv_len.data_ptr(),
                  n, T, max_q, hq, hkv, D, _CODE[dtype], code, _p(k_scale), _p(v_scale), n_pages, ps, stride,
                  block_table.shape[1], sm_scale, window, *beside, out.data_ptr(), lse.data_ptr(), workspace.data_ptr(),
                  workspace.nbytes, _p(error_word), _raw_stream(index))
    if rc:
        _check(rc, "kda_paged_attn")
    return out, lse
