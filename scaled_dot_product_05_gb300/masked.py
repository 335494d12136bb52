"""Attention whose rows see part of the keys: a sliding window with a few first
keys that stay visible (the Python side of sdpa_fwd_window and sdpa_bwd_window;
argument marshalling only)."""
from __future__ import annotations

import math

import torch

from . import _DTYPE, _lse_ptr, _shapes, _stream_ptr, bwd_workspace_bytes
from .cache import _alloc, _call, _empty_like, _like, _strides, _workspace
from ._abi import lib


def _dense(q, k, v):
    """(device, sizes) of the inputs of a call on tensors."""
    dev = q.get_device()
    if dev < 0:
        raise ValueError("tensors must be CUDA tensors")
    if q.dim() != 4 or k.dim() != 4 or k.shape != v.shape or k.shape[0] != q.shape[0] or k.shape[3] != q.shape[3]:
        raise ValueError("q must be [B, Sq, Hq, D], k and v [B, Skv, Hkv, D]")
    for t in (k, v):
        if t.get_device() != dev or t.dtype != q.dtype:
            raise ValueError("k and v must have q's dtype and be on its device")
    return dev, _shapes(q, k, v)


def sdpa_fwd_window(q, k, v, o=None, lse=None, *, window: int, sinks: int = 0, scale: float | None = None,
                    stream=None) -> torch.Tensor:
    """Causal attention with a sliding window: row i sees keys j <= i with
    j > i - window or j < sinks.

    q: [B, Sq, Hq, D], k and v: [B, Skv, Hkv, D], bf16 or fp16 views with a
    contiguous last dimension.  ``lse`` ([B, Hq, Sq] float32), when given,
    receives the log-sum-exp of every row's scores; a row that sees no key has
    -inf there and zeros in ``o``.  Returns ``o`` (allocated contiguous like q
    when not given)."""
    dev, (B, Hq, Hkv, Sq, Skv, D) = _dense(q, k, v)
    lo = None
    if o is None:
        o = _empty_like(q, stream, dev)
    else:
        lo = _like(o, q, dev, "o")
    if lse is not None and lse.get_device() != dev:
        raise ValueError("lse must be on the tensors' device")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _call(dev, lib().sdpa_fwd_window, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), _lse_ptr(lse, B, Hq, Sq), B,
          Hq, Hkv, Sq, Skv, D, _strides(q), _strides(k), _strides(v), lo, scale, window, sinks, _DTYPE.get(q.dtype, 99),
          _stream_ptr(stream, dev))
    return o


def sdpa_bwd_window(q, k, v, o, do, lse, dq=None, dk=None, dv=None, *, window: int, sinks: int = 0,
                    scale: float | None = None, workspace=None, stream=None):
    """Gradients (dq, dk, dv) of sum(do * o) for o = sdpa_fwd_window(q, k, v)
    with the same window, sinks and scale, on contiguous [B, S, H, D] tensors
    (D 64 or 128); ``lse`` is the forward's.  Outputs and the workspace
    (:func:`bwd_workspace_bytes`) are allocated when not given."""
    dev, (B, Hq, Hkv, Sq, Skv, D) = _dense(q, k, v)
    for t, name in ((o, "o"), (do, "do")):
        _like(t, q, dev, name)
    if lse is None or lse.get_device() != dev:
        raise ValueError("the forward's lse is required, on the tensors' device")
    dq = _empty_like(q, stream, dev) if dq is None else dq
    dk = _empty_like(k, stream, dev) if dk is None else dk
    dv = _empty_like(v, stream, dev) if dv is None else dv
    for t, like, name in ((dq, q, "dq"), (dk, k, "dk"), (dv, v, "dv")):
        _like(t, like, dev, name)
    for t in (q, k, v, o, do, dq, dk, dv):
        if not t.is_contiguous():
            raise ValueError("the backward pass takes contiguous tensors")
    if workspace is None:
        workspace = _alloc(stream, dev, q.new_empty, (bwd_workspace_bytes(B, Hq, Sq, D),), dtype=torch.uint8)
    ws, ws_bytes = _workspace(workspace, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    _call(dev, lib().sdpa_bwd_window, q.data_ptr(), k.data_ptr(), v.data_ptr(), o.data_ptr(), do.data_ptr(),
          _lse_ptr(lse, B, Hq, Sq), dq.data_ptr(), dk.data_ptr(), dv.data_ptr(), B, Hq, Hkv, Sq, Skv, D, scale, window,
          sinks, _DTYPE.get(q.dtype, 99), ws, ws_bytes, _stream_ptr(stream, dev))
    return dq, dk, dv
