"""Norm and rotation of queries and keys, the paged 8-bit cache and the
attention that reads it: the Python side of sdpa_qk_norm_rope,
sdpa_qk_norm_rope_bwd, sdpa_cache_append and sdpa_fwd_paged (argument
marshalling only)."""
from __future__ import annotations

import ctypes
import math

import torch

from . import _DTYPE, _layout, _lse_ptr, _run, _stream_ptr, _abi
from ._abi import lib

_WEIGHT_DTYPE = dict(_DTYPE)
_WEIGHT_DTYPE[torch.float32] = _abi.SDPA_DTYPE_F32


def rope_table(n_pos: int, rot_dim: int, *, base: float = 10000.0, device="cuda") -> torch.Tensor:
    """Rotation table [n_pos, rot_dim / 2, 2] (float32) of cosines and sines:
    pair i at position t turns by t * base^(-2 i / rot_dim), angles taken in
    64 bits.  Any other table of this shape (scaled positions or frequencies)
    serves as well."""
    inv = float(base) ** (-torch.arange(0, rot_dim, 2, dtype=torch.float64, device=device) / rot_dim)
    a = torch.arange(n_pos, dtype=torch.float64, device=device)[:, None] * inv
    return torch.stack((a.cos(), a.sin()), dim=-1).to(torch.float32)


def _on(device, *tensors):
    for t in tensors:
        if t is not None and t.device != device:
            raise ValueError("tensors must be on one CUDA device")


def _strides(t):
    """The tensor's layout argument: None where it is contiguous."""
    return None if t is None or t.is_contiguous() else ctypes.byref(_layout(t))


def _ptr(t):
    return None if t is None else t.data_ptr()


def _rope_arg(rope, interleaved, device):
    if rope is None:
        return None
    if rope.device != device or rope.dtype != torch.float32 or rope.dim() != 3 or rope.shape[2] != 2 \
            or not rope.is_contiguous():
        raise ValueError("rope must be a contiguous float32 table [n_pos, rot_dim / 2, 2] on the tensors' device")
    return ctypes.byref(_abi.Rope(rope.data_ptr(), rope.shape[0], 2 * rope.shape[1], int(bool(interleaved))))


def _int32(t, shape, device, name):
    if t is None:
        return None
    if t.device != device or t.dtype != torch.int32 or tuple(t.shape) != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on the tensors' device")
    return t.data_ptr()


def _weights(qw, kw, D, device):
    dt = None
    for w in (qw, kw):
        if w is None:
            continue
        if w.device != device or tuple(w.shape) != (D,) or not w.is_contiguous() or (dt is not None and w.dtype != dt):
            raise ValueError("weights must be contiguous [D] tensors of one dtype on the tensors' device")
        dt = w.dtype
    return _WEIGHT_DTYPE.get(dt, 99) if dt is not None else _abi.SDPA_DTYPE_F32


def _pair_shapes(q, k):
    if not q.is_cuda:
        raise ValueError("tensors must be CUDA tensors")
    if q.dim() != 4:
        raise ValueError("q must be [B, S, Hq, D]")
    B, S, Hq, D = q.shape
    if k is None:
        return B, S, Hq, 0, D
    if k.dim() != 4 or k.shape[:2] != q.shape[:2] or k.shape[3] != D or k.dtype != q.dtype:
        raise ValueError("k must be [B, S, Hkv, D] like q, with q's dtype")
    return B, S, Hq, k.shape[2], D


def _like(t, like, name):
    if t is not None and (like is None or t.shape != like.shape or t.dtype != like.dtype):
        raise ValueError(f"{name} must be shaped and typed like its input")


def sdpa_qk_norm_rope(q, k=None, q_out=None, k_out=None, *, norm: bool = True, q_weight=None, k_weight=None,
                      eps: float = 1e-6, rope=None, positions=None, interleaved: bool = False, stream=None):
    """Norm of queries and keys for each head and their rotation, in one pass:
    y = R(position) (x * w / sqrt(mean(x^2) + eps)) for every row of D channels.

    q: [B, S, Hq, D] and k: [B, S, Hkv, D] (or None), bf16 or fp16 views with
    a contiguous last dimension.  ``norm=False`` rotates only; ``rope`` is a
    table as :func:`rope_table` makes it (None: no rotation), ``positions``
    int32 [B, S] (None: 0 .. S - 1), weights [D] in float32 or q's dtype
    (None: ones).  Returns (q_out, k_out), allocated contiguous when not
    given; a tensor may be its own output."""
    B, S, Hq, Hkv, D = _pair_shapes(q, k)
    dev = q.device
    if q_out is None:
        q_out = torch.empty(q.shape, dtype=q.dtype, device=dev)
    if k_out is None and k is not None:
        k_out = torch.empty(k.shape, dtype=k.dtype, device=dev)
    _like(q_out, q, "q_out")
    _like(k_out, k, "k_out")
    _on(dev, k, q_out, k_out)
    _run(dev.index, lib().sdpa_qk_norm_rope, q.data_ptr(), _ptr(k), q_out.data_ptr(), _ptr(k_out), B, S, Hq, Hkv, D,
         _strides(q), _strides(k), _strides(q_out), _strides(k_out), int(bool(norm)), _ptr(q_weight), _ptr(k_weight),
         _weights(q_weight, k_weight, D, dev), float(eps), _rope_arg(rope, interleaved, dev),
         _int32(positions, (B, S), dev, "positions"), _DTYPE.get(q.dtype, 99), _stream_ptr(stream, dev.index))
    return q_out, k_out


def qk_norm_rope_bwd_workspace_bytes(B: int, S: int, Hq: int, Hkv: int, D: int) -> int:
    """Workspace bytes :func:`sdpa_qk_norm_rope_bwd` needs."""
    return int(lib().sdpa_qk_norm_rope_bwd_workspace_bytes(B, S, Hq, Hkv, D))


def sdpa_qk_norm_rope_bwd(q, k, dq_out, dk_out, dq=None, dk=None, *, norm: bool = True, q_weight=None, k_weight=None,
                          dq_weight=None, dk_weight=None, eps: float = 1e-6, rope=None, positions=None,
                          interleaved: bool = False, workspace=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of sum(dq_out * q_out) +
    sum(dk_out * k_out) for (q_out, k_out) = sdpa_qk_norm_rope(q, k, ...) with
    the same arguments.  The weights' gradients are float32 [D] (None without
    norm, and for an absent k); outputs and the workspace are allocated when
    not given."""
    B, S, Hq, Hkv, D = _pair_shapes(q, k)
    dev = q.device
    if (k is None) != (dk_out is None):
        raise ValueError("k and dk_out go together")
    if dq_out is None:
        raise ValueError("dq_out is required")
    dq = torch.empty(q.shape, dtype=q.dtype, device=dev) if dq is None else dq
    if k is not None and dk is None:
        dk = torch.empty(k.shape, dtype=k.dtype, device=dev)
    _like(dq, q, "dq")
    _like(dk, k, "dk")
    _like(dq_out, q, "dq_out")
    _like(dk_out, k, "dk_out")
    if norm:
        if dq_weight is None:
            dq_weight = torch.empty(D, dtype=torch.float32, device=dev)
        if dk_weight is None and k is not None:
            dk_weight = torch.empty(D, dtype=torch.float32, device=dev)
        if workspace is None:
            workspace = torch.empty(qk_norm_rope_bwd_workspace_bytes(B, S, Hq, Hkv, D), dtype=torch.uint8, device=dev)
    else:
        dq_weight = dk_weight = None
    if k is None and dk_weight is not None:
        raise ValueError("dk_weight without k")
    for t in (dq_weight, dk_weight):
        if t is not None and (t.dtype != torch.float32 or tuple(t.shape) != (D,) or not t.is_contiguous()):
            raise ValueError("weight gradients must be contiguous float32 [D] tensors")
    if workspace is not None and not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _on(dev, k, dq_out, dk_out, dq, dk, dq_weight, dk_weight, workspace)
    _run(dev.index, lib().sdpa_qk_norm_rope_bwd, q.data_ptr(), _ptr(k), dq_out.data_ptr(), _ptr(dk_out), dq.data_ptr(),
         _ptr(dk), _ptr(dq_weight), _ptr(dk_weight), B, S, Hq, Hkv, D, _strides(q), _strides(k), _strides(dq_out),
         _strides(dk_out), _strides(dq), _strides(dk), int(bool(norm)), _ptr(q_weight), _ptr(k_weight),
         _weights(q_weight, k_weight, D, dev), float(eps), _rope_arg(rope, interleaved, dev),
         _int32(positions, (B, S), dev, "positions"), _DTYPE.get(q.dtype, 99), _ptr(workspace),
         0 if workspace is None else workspace.numel() * workspace.element_size(), _stream_ptr(stream, dev.index))
    return dq, dk, dq_weight, dk_weight


class PagedCache:
    """A paged key / value cache in 8 bits: E4M3 codes ``k`` and ``v``
    [n_pages, page_size, Hkv, D] (views with a contiguous last dimension) and
    one float32 scale for each page and KV head, ``k_scale`` and ``v_scale``
    [n_pages, Hkv]; a value is code * scale.  The tensors are the caller's and
    may be read and copied as such; their addresses are taken here once."""

    def __init__(self, k: torch.Tensor, v: torch.Tensor, k_scale: torch.Tensor, v_scale: torch.Tensor):
        for t in (k, v):
            if not t.is_cuda or t.dim() != 4 or t.dtype not in (torch.float8_e4m3fn, torch.uint8) or t.shape != k.shape \
                    or t.device != k.device or t.stride(3) != 1:
                raise ValueError("k and v must be E4M3 CUDA tensors [n_pages, page_size, Hkv, D] with a contiguous "
                                 "last dimension")
        for t in (k_scale, v_scale):
            if t.device != k.device or t.dtype != torch.float32 or tuple(t.shape) != (k.shape[0], k.shape[2]) \
                    or not t.is_contiguous():
                raise ValueError("scales must be contiguous float32 tensors [n_pages, Hkv] on the codes' device")
        self.k, self.v, self.k_scale, self.v_scale = k, v, k_scale, v_scale
        self.n_pages, self.page_size, self.n_heads, self.head_dim = k.shape
        self._layouts = (_layout(k), _layout(v))
        self._c = _abi.Cache(k.data_ptr(), v.data_ptr(), k_scale.data_ptr(), v_scale.data_ptr(), self.n_pages,
                             self.page_size, ctypes.pointer(self._layouts[0]), ctypes.pointer(self._layouts[1]))
        self._ref = ctypes.byref(self._c)

    @classmethod
    def empty(cls, n_pages: int, page_size: int, n_heads: int, head_dim: int, device="cuda") -> "PagedCache":
        """A cache with nothing in it, each head's part of a page contiguous
        (the layout that the attention reads in the longest runs)."""
        def codes():
            t = torch.zeros((n_pages, n_heads, page_size, head_dim), dtype=torch.uint8, device=device)
            return t.view(torch.float8_e4m3fn).permute(0, 2, 1, 3)

        def scales():
            return torch.ones((n_pages, n_heads), dtype=torch.float32, device=device)
        return cls(codes(), codes(), scales(), scales())


def _cache_args(cache, block_table, start, count, B):
    dev = cache.k.device
    if block_table.dim() != 2:
        raise ValueError("block_table must be [B, max_pages]")
    width = block_table.shape[1]
    return (_int32(block_table, (B, width), dev, "block_table"), _int32(start, (B,), dev, "start"),
            _int32(count, (B,), dev, "count"), width)


def sdpa_cache_append(k, v, cache: PagedCache, block_table, start, count=None, *, rope=None, interleaved: bool = False,
                      stream=None) -> None:
    """Appends k and v ([B, S, Hkv, D], bf16 or fp16) to the cache, the keys
    rotated by their positions on the way.  Token i < count[b] of sequence b
    goes to position start[b] + i: page block_table[b, position / page_size].
    block_table (int32 [B, max_pages]), start and count (int32 [B]; None: S
    tokens each) are CUDA tensors; nothing is read back to the host."""
    dev = cache.k.device
    if k.dim() != 4 or k.shape != v.shape or k.dtype != v.dtype:
        raise ValueError("k and v must be [B, S, Hkv, D] tensors of one shape and dtype")
    B, S, Hkv, D = k.shape
    if Hkv != cache.n_heads or D != cache.head_dim:
        raise ValueError("k and v must have the cache's heads and head dimension")
    _on(dev, k, v)
    table_p, start_p, count_p, width = _cache_args(cache, block_table, start, count, B)
    _run(dev.index, lib().sdpa_cache_append, k.data_ptr(), v.data_ptr(), cache._ref, table_p, start_p, count_p, B, S, Hkv,
         D, width, _strides(k), _strides(v), _rope_arg(rope, interleaved, dev), _DTYPE.get(k.dtype, 99),
         _stream_ptr(stream, dev.index))


def paged_workspace_bytes(B: int, Hq: int, Hkv: int, Sq: int, D: int) -> int:
    """Workspace bytes :func:`sdpa_fwd_paged` needs."""
    return int(lib().sdpa_paged_workspace_bytes(B, Hq, Hkv, Sq, D))


def sdpa_fwd_paged(q, cache: PagedCache, block_table, start, count=None, o=None, lse=None, *, causal: bool = True,
                   scale: float | None = None, workspace=None, stream=None) -> torch.Tensor:
    """Attention of q ([B, Sq, Hq, D], bf16 or fp16) over the cache.  Query
    i < count[b] of sequence b stands at position start[b] + i, as in
    :func:`sdpa_cache_append`, and sees positions 0 .. start[b] + i (causal) or
    all 0 .. start[b] + count[b] - 1.  Rows behind count[b] of ``o`` and
    ``lse`` ([B, Hq, Sq] float32) are left as they are.  ``o`` (like q) and
    the workspace are allocated when not given.  Returns ``o``."""
    dev = cache.k.device
    if q.dim() != 4 or q.shape[3] != cache.head_dim:
        raise ValueError("q must be [B, Sq, Hq, D] with the cache's head dimension")
    B, Sq, Hq, D = q.shape
    Hkv = cache.n_heads
    if o is None:
        o = torch.empty(q.shape, dtype=q.dtype, device=dev)
    _like(o, q, "o")
    if workspace is None:
        workspace = torch.empty(paged_workspace_bytes(B, Hq, Hkv, Sq, D), dtype=torch.uint8, device=dev)
    elif not workspace.is_contiguous():
        raise ValueError("workspace must be contiguous")
    _on(dev, q, o, lse, workspace)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    table_p, start_p, count_p, width = _cache_args(cache, block_table, start, count, B)
    _run(dev.index, lib().sdpa_fwd_paged, q.data_ptr(), cache._ref, table_p, start_p, count_p, o.data_ptr(),
         _lse_ptr(lse, B, Hq, Sq), B, Hq, Hkv, Sq, D, width, _strides(q), _strides(o), float(scale), int(bool(causal)),
         _DTYPE.get(q.dtype, 99), workspace.data_ptr(), workspace.numel() * workspace.element_size(),
         _stream_ptr(stream, dev.index))
    return o
