"""Norm and rotation of queries and keys, the paged 8-bit cache and the
attention that reads it: the Python side of sdpa_qk_norm_rope,
sdpa_qk_norm_rope_bwd, sdpa_cache_append and sdpa_fwd_paged (argument
marshalling only)."""
from __future__ import annotations

import ctypes
import functools
import math

import torch

from . import _DTYPE, _layout, _lse_ptr, _run, _stream_ptr, _abi
from ._abi import check, lib

_DENSE = torch.contiguous_format
_lib = None


def _bound():
    """The loaded library, kept here after the first call."""
    global _lib
    _lib = lib()
    return _lib


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


# A decoding step makes a few such calls for each layer, and their kernels run
# for a few microseconds: the checks below read each tensor attribute once and
# compare device numbers instead of device objects.

_get_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)


def _call(device: int, fn, *args) -> None:
    """Calls the library with the tensors' device current."""
    if _get_device() == device:
        status = fn(*args)
        if status:
            check(status)
    else:
        _run(device, fn, *args)


def _alloc(stream, dev, make, /, *args, **kwargs):
    """make(...) in the memory pool of the stream that the call runs on: what
    the call leaves behind (a workspace) or takes over from earlier work is
    then ordered by that stream."""
    if stream is None:                                 # the current one
        return make(*args, **kwargs)
    if not isinstance(stream, torch.cuda.Stream):
        handle = stream.cuda_stream if hasattr(stream, "cuda_stream") else int(stream)
        stream = torch.cuda.ExternalStream(handle, dev) if handle else torch.cuda.default_stream(dev)
    with torch.cuda.stream(stream):
        return make(*args, **kwargs)


def _empty_like(t, stream, dev):
    if stream is None:
        return torch.empty_like(t, memory_format=_DENSE)
    return _alloc(stream, dev, torch.empty_like, t, memory_format=_DENSE)


@functools.lru_cache(maxsize=1024)
def _layout_ref(strides):
    """sdpa_layout_t of a 4-D tensor's strides, by value."""
    if len(strides) != 4 or strides[3] != 1:
        raise ValueError("tensors must be 4-D [B, S, H, D] views with a contiguous last dimension")
    return ctypes.byref(_abi.Layout(*strides[:3]))


def _strides(t):
    """The tensor's layout argument: None where it is contiguous."""
    return None if t.is_contiguous() else _layout_ref(t.stride())


def _like(t, like, device, name):
    """The layout argument of an output (or gradient) that the caller gave."""
    if t.shape != like.shape or t.dtype != like.dtype or t.get_device() != device:
        raise ValueError(f"{name} must be shaped and typed like its input, on its device")
    return _strides(t)


def _rope_arg(rope, interleaved, device):
    if rope is None:
        return None
    shape = rope.shape
    if rope.get_device() != device or rope.dtype != torch.float32 or len(shape) != 3 or shape[2] != 2 \
            or not rope.is_contiguous():
        raise ValueError("rope must be a contiguous float32 table [n_pos, rot_dim / 2, 2] on the tensors' device")
    return ctypes.byref(_abi.Rope(rope.data_ptr(), shape[0], 2 * shape[1], 1 if interleaved else 0))


def _int32(t, shape, device, name):
    if t is None:
        return None
    if t.get_device() != device or t.dtype != torch.int32 or t.shape != shape or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 tensor {list(shape)} on the tensors' device")
    return t.data_ptr()


def _weights(qw, kw, D, device):
    """(address, address, dtype code) of the norm's weights."""
    code, ptrs = _abi.SDPA_DTYPE_F32, [None, None]
    for i, w in enumerate((qw, kw)):
        if w is None:
            continue
        if w.get_device() != device or w.shape != (D,) or not w.is_contiguous() or \
                (i and qw is not None and w.dtype != qw.dtype):
            raise ValueError("weights must be contiguous [D] tensors of one dtype on the tensors' device")
        code, ptrs[i] = _WEIGHT_DTYPE.get(w.dtype, 99), w.data_ptr()
    return ptrs[0], ptrs[1], code


def _pair_shapes(q, k):
    """(device, B, S, Hq, Hkv, D, layout arguments of q and k) of a pair of inputs."""
    device = q.get_device()
    if device < 0:
        raise ValueError("tensors must be CUDA tensors")
    shape = q.shape
    if len(shape) != 4:
        raise ValueError("q must be [B, S, Hq, D]")
    B, S, Hq, D = shape
    if k is None:
        return device, B, S, Hq, 0, D, _strides(q), None
    kshape = k.shape
    if len(kshape) != 4 or kshape[0] != B or kshape[1] != S or kshape[3] != D or k.dtype != q.dtype \
            or k.get_device() != device:
        raise ValueError("k must be [B, S, Hkv, D] like q, with q's dtype, on its device")
    return device, B, S, Hq, kshape[2], D, _strides(q), _strides(k)


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
    dev, B, S, Hq, Hkv, D, lq, lk = _pair_shapes(q, k)
    lqo = lko = kp = kop = None
    if q_out is None:
        q_out = _empty_like(q, stream, dev)
    else:
        lqo = _like(q_out, q, dev, "q_out")
    if k is not None:
        if k_out is None:
            k_out = _empty_like(k, stream, dev)
        else:
            lko = _like(k_out, k, dev, "k_out")
        kp, kop = k.data_ptr(), k_out.data_ptr()
    elif k_out is not None:
        raise ValueError("k_out without k")
    qw, kw, wdt = _weights(q_weight, k_weight, D, dev)
    _call(dev, (_lib or _bound()).sdpa_qk_norm_rope, q.data_ptr(), kp, q_out.data_ptr(), kop, B, S, Hq, Hkv, D, lq, lk, lqo,
          lko, 1 if norm else 0, qw, kw, wdt, eps, _rope_arg(rope, interleaved, dev),
          _int32(positions, (B, S), dev, "positions"), _DTYPE.get(q.dtype, 99), _stream_ptr(stream, dev))
    return q_out, k_out


def qk_norm_rope_bwd_workspace_bytes(B: int, S: int, Hq: int, Hkv: int, D: int) -> int:
    """Workspace bytes :func:`sdpa_qk_norm_rope_bwd` needs."""
    return int(lib().sdpa_qk_norm_rope_bwd_workspace_bytes(B, S, Hq, Hkv, D))


def _weight_grad(t, D, device):
    if t.dtype != torch.float32 or t.shape != (D,) or not t.is_contiguous() or t.get_device() != device:
        raise ValueError("weight gradients must be contiguous float32 [D] tensors on the tensors' device")
    return t.data_ptr()


def _workspace(t, device):
    if t.get_device() != device or not t.is_contiguous():
        raise ValueError("workspace must be a contiguous tensor on the tensors' device")
    return t.data_ptr(), t.numel() * t.element_size()


def sdpa_qk_norm_rope_bwd(q, k, dq_out, dk_out, dq=None, dk=None, *, norm: bool = True, q_weight=None, k_weight=None,
                          dq_weight=None, dk_weight=None, eps: float = 1e-6, rope=None, positions=None,
                          interleaved: bool = False, workspace=None, stream=None):
    """Gradients (dq, dk, dq_weight, dk_weight) of sum(dq_out * q_out) +
    sum(dk_out * k_out) for (q_out, k_out) = sdpa_qk_norm_rope(q, k, ...) with
    the same arguments.  The weights' gradients are float32 [D] (None without
    norm, and for an absent k); outputs and the workspace are allocated when
    not given."""
    dev, B, S, Hq, Hkv, D, lq, lk = _pair_shapes(q, k)
    if dq_out is None or (k is None) != (dk_out is None):
        raise ValueError("dq_out is required; k and dk_out go together")
    if k is None and (dk is not None or dk_weight is not None):
        raise ValueError("dk and dk_weight without k")
    lgq = _like(dq_out, q, dev, "dq_out")
    ldq = ldk = lgk = kp = gkp = dkp = dwq = dwk = ws = None
    ws_bytes = 0
    if dq is None:
        dq = _empty_like(q, stream, dev)
    else:
        ldq = _like(dq, q, dev, "dq")
    if k is not None:
        lgk = _like(dk_out, k, dev, "dk_out")
        if dk is None:
            dk = _empty_like(k, stream, dev)
        else:
            ldk = _like(dk, k, dev, "dk")
        kp, gkp, dkp = k.data_ptr(), dk_out.data_ptr(), dk.data_ptr()
    if norm:
        if dq_weight is None:
            dq_weight = _alloc(stream, dev, torch.empty, D, dtype=torch.float32, device=dev)
        dwq = _weight_grad(dq_weight, D, dev)
        if k is not None:
            if dk_weight is None:
                dk_weight = _alloc(stream, dev, torch.empty, D, dtype=torch.float32, device=dev)
            dwk = _weight_grad(dk_weight, D, dev)
        if workspace is None:
            workspace = _alloc(stream, dev, q.new_empty, (qk_norm_rope_bwd_workspace_bytes(B, S, Hq, Hkv, D),),
                               dtype=torch.uint8)
        ws, ws_bytes = _workspace(workspace, dev)
    else:
        dq_weight = dk_weight = None
    qw, kw, wdt = _weights(q_weight, k_weight, D, dev)
    _call(dev, (_lib or _bound()).sdpa_qk_norm_rope_bwd, q.data_ptr(), kp, dq_out.data_ptr(), gkp, dq.data_ptr(), dkp, dwq,
          dwk, B, S, Hq, Hkv, D, lq, lk, lgq, lgk, ldq, ldk, 1 if norm else 0, qw, kw, wdt, eps,
          _rope_arg(rope, interleaved, dev), _int32(positions, (B, S), dev, "positions"), _DTYPE.get(q.dtype, 99), ws,
          ws_bytes, _stream_ptr(stream, dev))
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
        self._device = k.get_device()

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
    dev = cache._device
    shape = block_table.shape
    if len(shape) != 2:
        raise ValueError("block_table must be [B, max_pages]")
    return (_int32(block_table, (B, shape[1]), dev, "block_table"), _int32(start, (B,), dev, "start"),
            _int32(count, (B,), dev, "count"), shape[1])


def sdpa_cache_append(k, v, cache: PagedCache, block_table, start, count=None, *, rope=None, interleaved: bool = False,
                      stream=None) -> None:
    """Appends k and v ([B, S, Hkv, D], bf16 or fp16) to the cache, the keys
    rotated by their positions on the way.  Token i < count[b] of sequence b
    goes to position start[b] + i: page block_table[b, position / page_size].
    block_table (int32 [B, max_pages]), start and count (int32 [B]; None: S
    tokens each) are CUDA tensors; nothing is read back to the host.  A
    sequence with a negative start is left out as a whole and reported by
    :func:`sdpa_device_error`, as are indexes out of range."""
    dev = cache._device
    shape = k.shape
    if len(shape) != 4 or v.shape != shape or k.dtype != v.dtype:
        raise ValueError("k and v must be [B, S, Hkv, D] tensors of one shape and dtype")
    B, S, Hkv, D = shape
    if Hkv != cache.n_heads or D != cache.head_dim:
        raise ValueError("k and v must have the cache's heads and head dimension")
    if k.get_device() != dev or v.get_device() != dev:
        raise ValueError("k and v must be on the cache's device")
    table_p, start_p, count_p, width = _cache_args(cache, block_table, start, count, B)
    _call(dev, (_lib or _bound()).sdpa_cache_append, k.data_ptr(), v.data_ptr(), cache._ref, table_p, start_p, count_p, B, S,
          Hkv, D, width, _strides(k), _strides(v), _rope_arg(rope, interleaved, dev), _DTYPE.get(k.dtype, 99),
          _stream_ptr(stream, dev))


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
    the workspace are allocated when not given, from ``stream``'s memory.
    Returns ``o``."""
    dev = cache._device
    shape = q.shape
    if len(shape) != 4 or shape[3] != cache.head_dim:
        raise ValueError("q must be [B, Sq, Hq, D] with the cache's head dimension")
    if q.get_device() != dev:
        raise ValueError("q must be on the cache's device")
    B, Sq, Hq, D = shape
    Hkv = cache.n_heads
    lo = None
    if o is None:
        o = _empty_like(q, stream, dev)
    else:
        lo = _like(o, q, dev, "o")
    if lse is not None and lse.get_device() != dev:
        raise ValueError("lse must be on the cache's device")
    if workspace is None:
        workspace = _alloc(stream, dev, q.new_empty, (paged_workspace_bytes(B, Hq, Hkv, Sq, D),), dtype=torch.uint8)
    ws, ws_bytes = _workspace(workspace, dev)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    table_p, start_p, count_p, width = _cache_args(cache, block_table, start, count, B)
    _call(dev, (_lib or _bound()).sdpa_fwd_paged, q.data_ptr(), cache._ref, table_p, start_p, count_p, o.data_ptr(),
          _lse_ptr(lse, B, Hq, Sq), B, Hq, Hkv, Sq, D, width, _strides(q), lo, scale, 1 if causal else 0,
          _DTYPE.get(q.dtype, 99), ws, ws_bytes, _stream_ptr(stream, dev))
    return o
