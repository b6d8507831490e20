"""Binding of the verification of drafted tokens (include/kda.h).

As in ``paged.py``, argument marshalling only, with the compiled way first.
"""
from __future__ import annotations

import torch

from . import paged
from .kda import KDAError, _check
from .paged import _CODE, _F32, _I32, _fit, _ints, _p, _raw_stream, _typed

DEVERR_TOKEN, DEVERR_PROBS = 64, 128


def _rows(name, t, n, w, v, dtype, index):
    """A [n, w, v] tensor whose rows may lie apart; returns the strides of its first two dimensions."""
    if t.shape != (n, w, v) or t.dtype is not dtype:
        raise KDAError(f"{name} must be {[n, w, v]}, of target's dtype")
    if t.get_device() != index or index < 0:
        raise KDAError("all tensors must be CUDA tensors on one device")
    a = t.stride()
    if t.is_contiguous():
        return w * v, v
    if v > 1 and a[2] != 1:
        raise KDAError(f"each row of {name} must be contiguous (rows may lie apart)")
    return (a[0] if n > 1 else 0), (a[1] if w > 1 else max(v, a[1]))


def verify_drafts_workspace_size(n: int, W: int, vocabulary: int, dtype=torch.float32) -> int:
    """Bytes of workspace that verify_drafts needs for up to n requests (0 for shapes it does not take)."""
    if dtype not in _CODE or not (_fit(n) and _fit(W) and _fit(vocabulary)):
        return 0
    return int((paged._declared or paged._lib()).kda_verify_drafts_workspace_size(n, W, vocabulary, _CODE[dtype]))


def verify_drafts(target, draft_tokens, uniforms, draft=None, n_draft=None, workspace=None, error_word=None):
    """kda_verify_drafts: target [n, W, vocabulary] float32 or bfloat16 probabilities
    (row j: after j drafts), draft_tokens int32 [n, W - 1], uniforms float32 [n, W] in
    [0, 1); draft [n, W - 1, vocabulary], the probabilities the drafts were drawn from
    (None: the drafts are certain); n_draft int32 [n], drafts of each request (None: W - 1).
    Returns (num_accepted int32 [n], tokens int32 [n, W]: the accepted drafts, the
    token after them, then -1)."""
    done = paged._fast_verify(target, draft_tokens, uniforms, draft, n_draft, workspace, error_word)
    if done is not None:
        return done
    lib = paged._declared or paged._lib()
    index = target.get_device()
    if target.dim() != 3 or target.dtype not in _CODE:
        raise KDAError("target must be [n, W, vocabulary], float32 or bfloat16")
    n, w, v = target.shape
    _ints("n W vocabulary", n, w, v)
    ts, tr = _rows("target", target, n, w, v, target.dtype, index)
    ds, dr = (0, 0) if draft is None else _rows("draft", draft, n, w - 1, v, target.dtype, index)
    for t in (draft_tokens, uniforms, n_draft, workspace, error_word):
        if t is not None and (t.get_device() != index or not t.is_contiguous()):
            raise KDAError("all tensors must be contiguous CUDA tensors on one device")
    _typed(_I32, "draft_tokens n_draft error_word", draft_tokens, n_draft, error_word)
    _typed(_F32, "uniforms", uniforms)
    if draft_tokens.shape != (n, w - 1) or uniforms.shape != (n, w) or (n_draft is not None and n_draft.numel() != n):
        raise KDAError("draft_tokens must be [n, W - 1], uniforms [n, W] and n_draft [n]")
    accepted, tokens = draft_tokens.new_empty(n), draft_tokens.new_empty(n, w)
    if w == 1:
        draft = None
    if workspace is None:
        workspace = draft_tokens.new_empty(verify_drafts_workspace_size(n, w, v, target.dtype), dtype=torch.uint8)
    with torch.cuda.device(index):
        rc = lib.kda_verify_drafts(target.data_ptr(), _p(draft), draft_tokens.data_ptr() or None, uniforms.data_ptr(),
                                   _p(n_draft), n, w, v, _CODE[target.dtype], ts, tr, ds, dr, accepted.data_ptr(),
                                   tokens.data_ptr(), workspace.data_ptr(), workspace.nbytes, _p(error_word), _raw_stream(index))
    if rc:
        _check(rc, "kda_verify_drafts")
    return accepted, tokens
