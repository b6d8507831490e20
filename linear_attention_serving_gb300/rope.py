"""Binding of the rotary positions and per-head norms (include/kda.h): alone, and
joined with the append of keys and values into the paged cache.

As in ``paged.py``, argument marshalling only, with the compiled way first.
"""
from __future__ import annotations

import ctypes

import torch

from . import paged
from .kda import D, KDAError, _check
from .paged import _CODE, _F32, _I32, _I64, _cache, _ints, _p, _raw_stream, _typed

SCALINGS = {"none": 0, "linear": 1, "ntk": 2, "yarn": 3}


def rope_frequencies(rot_dim, base=10000.0, scaling="none", factor=1.0, original_len=0, beta_fast=32.0, beta_slow=1.0,
                     device=None):
    """kda_rope_frequencies: (freq int64 [rot_dim / 2] on `device`, amplitude), once per
    model.  scaling: "none", "linear", "ntk" or "yarn" (contexts stretched by `factor`).
    "yarn" is the ramp of the paper's text, over a pair's turns; checkpoints trained with the
    ramp over the pair's number take a table of their own, round(f_i / 2 pi * 2^64) in int64."""
    if scaling not in SCALINGS:
        raise KDAError(f"unsupported scaling {scaling!r}: one of {', '.join(SCALINGS)}")
    _ints("rot_dim", rot_dim)
    lib = paged._declared or paged._lib()
    freq = torch.empty(max(0, rot_dim // 2), dtype=_I64)
    amplitude = ctypes.c_float()
    rc = lib.kda_rope_frequencies(rot_dim, base, SCALINGS[scaling], factor, original_len, beta_fast, beta_slow,
                                  freq.data_ptr(), ctypes.byref(amplitude))
    if rc:
        _check(rc, "kda_rope_frequencies")
    # (once per model: the copy is waited for, so that any stream may read the table)
    return freq if device is None else freq.to(device), amplitude.value


def _rows(name, t, index, shape=None, dtype=None):
    """A [T, heads, 128] tensor whose tokens may lie apart; returns their stride."""
    if t.dim() != 3 or t.shape[2] != D or (shape is not None and t.shape != shape):
        raise KDAError(f"{name} must be [T, heads, 128]" if shape is None else f"{name} must be {list(shape)}")
    if t.get_device() != index or index < 0:
        raise KDAError("all tensors must be CUDA tensors on one device")
    if dtype is not None and t.dtype is not dtype:
        raise KDAError(f"{name} must have q's dtype")
    T, h, _ = t.shape
    if t.is_contiguous():
        return h * D
    a = t.stride()
    if a[2] != 1 or (h > 1 and a[1] != D):
        raise KDAError(f"each token of {name} must be contiguous (tokens may lie apart)")
    return a[0] if T > 1 else max(a[0], h * D)


def _common(q, k, positions, freq, q_weight, k_weight, q_out, index):
    if q.dtype not in _CODE:
        raise KDAError(f"unsupported dtype {q.dtype}: q and k must be bfloat16 or float32")
    qs, ks = _rows("q", q, index), _rows("k", k, index, dtype=q.dtype)
    T = q.shape[0]
    if positions is None and freq is not None and freq.numel() > 0:
        raise KDAError("positions may be None only without a rotation")
    if k.shape[0] != T or (positions is not None and positions.numel() != T):
        raise KDAError("q and k must be [T, heads, 128], positions [T]")
    _ints("Hq Hkv rot_dim", q.shape[1], k.shape[1], 0 if freq is None else 2 * freq.numel())
    for t in (positions, freq, q_weight, k_weight):
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            raise KDAError("all tensors must be contiguous CUDA tensors on one device")
    _typed(_I32, "positions", positions)
    _typed(_I64, "freq", freq)
    _typed(_F32, "q_weight k_weight", q_weight, k_weight)
    for name, t in (("q_weight", q_weight), ("k_weight", k_weight)):
        if t is not None and t.numel() != D:
            raise KDAError(f"{name} must be [128]")
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=q.device)
    return qs, ks, q_out, _rows("q_out", q_out, index, q.shape, q.dtype)


def qk_rope(q, k, positions, freq, amplitude=1.0, interleaved=False, q_weight=None, k_weight=None, eps=1e-6, q_out=None,
            k_out=None):
    """kda_qk_rope: q [T, Hq, 128] and k [T, Hkv, 128] (parts of one projection, say)
    normed for each head where a weight float32 [128] is given, and turned by
    positions int32 [T].  freq and amplitude from rope_frequencies; freq None: no
    rotation (positions may be None then).  Returns (q_out, k_out), which may be q and k
    themselves."""
    done = paged._fast_rope(q, k, positions, freq, amplitude, interleaved, q_weight, k_weight, eps, q_out, k_out)
    if done is not None:
        return done
    lib = paged._declared or paged._lib()
    index = q.get_device()
    qs, ks, q_out, qos = _common(q, k, positions, freq, q_weight, k_weight, q_out, index)
    if k_out is None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=k.device)
    kos = _rows("k_out", k_out, index, k.shape, q.dtype)
    with torch.cuda.device(index):
        rc = lib.kda_qk_rope(q.data_ptr(), k.data_ptr(), _p(positions), _p(freq), amplitude, _p(q_weight), _p(k_weight),
                             eps, q.shape[0], q.shape[1], k.shape[1], D, 0 if freq is None else 2 * freq.numel(),
                             int(interleaved), _CODE[q.dtype], qs, ks, q_out.data_ptr(), k_out.data_ptr(), qos, kos,
                             _raw_stream(index))
    if rc:
        _check(rc, "kda_qk_rope")
    return q_out, k_out


def paged_rope_append(q, k, v, positions, slot_map, freq, k_cache, v_cache, amplitude=1.0, interleaved=False, q_weight=None,
                      k_weight=None, eps=1e-6, k_scale=None, v_scale=None, q_out=None, error_word=None):
    """kda_paged_rope_append: qk_rope with the keys, and the values v [T, Hkv, 128],
    written into the caches at slot_map, as paged_append does.  Returns q_out."""
    done = paged._fast_rope_append(q, k, v, positions, slot_map, freq, k_cache, v_cache, amplitude, interleaved, q_weight,
                                   k_weight, eps, k_scale, v_scale, q_out, error_word)
    if done is not None:
        return done
    lib = paged._declared or paged._lib()
    index = q.get_device()
    qs, ks, q_out, qos = _common(q, k, positions, freq, q_weight, k_weight, q_out, index)
    vs = _rows("v", v, index, k.shape, q.dtype)
    n, h, ps, stride, code = _cache(index, k_cache, v_cache, k_scale, v_scale)
    if k.shape[1] != h:
        raise KDAError("k and v must have the caches' kv heads")
    for t in (slot_map, k_scale, v_scale, error_word):
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            raise KDAError("all tensors must be contiguous CUDA tensors on one device")
    _typed(_I64, "slot_map", slot_map)
    _typed(_I32, "error_word", error_word)
    if slot_map.numel() != q.shape[0]:
        raise KDAError("slot_map must be [T]")
    with torch.cuda.device(index):
        rc = lib.kda_paged_rope_append(q.data_ptr(), k.data_ptr(), v.data_ptr(), _p(positions), slot_map.data_ptr(),
                                       _p(freq), amplitude, _p(q_weight), _p(k_weight), eps, q.shape[0], q.shape[1], h, D,
                                       0 if freq is None else 2 * freq.numel(), int(interleaved), _CODE[q.dtype], code, qs, ks,
                                       vs, q_out.data_ptr(), qos, _p(k_scale), _p(v_scale), k_cache.data_ptr(),
                                       v_cache.data_ptr(), n, ps, stride, _p(error_word), _raw_stream(index))
    if rc:
        _check(rc, "kda_paged_rope_append")
    return q_out
