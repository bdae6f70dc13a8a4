"""Paged 8-bit key/value cache: binding of the calls in ``include/mhc_kv.h``.

    kv_cache(num_pages, heads, page_tokens, head_dim) -> dict
    kv_append(cache, k, v, block_table, seq_lens, cu_q=None, q=None, cos=None, sin=None, ...) -> Tensor | None
    kv_attend(q, cache, block_table, seq_lens, cu_q=None, ...) -> dict

A cache is a dict of tensors: "k", "v" float8_e4m3fn [num_pages, heads,
page_tokens, head_dim] and "k_scale", "v_scale" fp32 [num_pages, heads].
block_table int32 [B, width] holds each sequence's pages, seq_lens int32 [B]
each sequence's length with its new tokens, cu_q int32 [B + 1] where each
sequence's new tokens begin (None: one for each sequence).  The calls are
asynchronous; a bad index on the device is reported by ``device_status()``.
"""
from __future__ import annotations

import ctypes
import math

import torch

from . import _check, _dev_ptr, _device_index, _stream_ptr, _workspaces, load_library

__all__ = ["kv_cache", "kv_append", "kv_attend", "kv_workspace_for"]


class _Cache(ctypes.Structure):
    """mhc_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("heads", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("head_dim", ctypes.c_int)]


def declare(lib) -> None:
    """Argument types of the kv entry points (called once by ``load_library``)."""
    P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    C = ctypes.POINTER(_Cache)
    lib.mhc_kv_append.argtypes = [C, P, I64, P, I64, P, I64, I, P, I64, P, P, I64, I, I, P, I64, P, P, I64, I64, P]
    lib.mhc_kv_append.restype = I
    lib.mhc_kv_attend.argtypes = [C, P, I64, I, P, I64, P, P, I64, I64, F, P, P, P, ctypes.c_size_t, P]
    lib.mhc_kv_attend.restype = I
    lib.mhc_kv_attend_workspace_bytes.argtypes = [C, I, I64, I64]
    lib.mhc_kv_attend_workspace_bytes.restype = ctypes.c_size_t


def kv_cache(num_pages: int, heads: int, page_tokens: int = 64, head_dim: int = 128, *, device="cuda") -> dict:
    """An empty cache of one layer (every code and scale zero)."""
    shape = (num_pages, heads, page_tokens, head_dim)
    return {"k": torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
            "v": torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
            "k_scale": torch.zeros(num_pages, heads, dtype=torch.float32, device=device),
            "v_scale": torch.zeros(num_pages, heads, dtype=torch.float32, device=device)}


def _cache_arg(cache: dict) -> tuple[_Cache, torch.device]:
    k = cache["k"]
    if k.dim() != 4:
        raise ValueError("cache['k'] must be [num_pages, heads, page_tokens, head_dim]")
    pages, heads, tokens, dim = k.shape
    dev = k.device
    if cache["v"].shape != k.shape:
        raise ValueError("cache['k'] and cache['v'] must have the same shape")
    for n in ("k_scale", "v_scale"):
        if tuple(cache[n].shape) != (pages, heads):
            raise ValueError(f"cache['{n}'] must be [num_pages, heads]")
    return _Cache(_dev_ptr(k, "cache['k']", torch.float8_e4m3fn, dev),
                  _dev_ptr(cache["v"], "cache['v']", torch.float8_e4m3fn, dev),
                  _dev_ptr(cache["k_scale"], "cache['k_scale']", torch.float32, dev),
                  _dev_ptr(cache["v_scale"], "cache['v_scale']", torch.float32, dev), pages, heads, tokens, dim), dev


def _rows_arg(t: torch.Tensor, name: str, dim: int, dev) -> tuple[int, int, int, int]:
    """Pointer, token stride, tokens and heads of a bf16 [T, heads, head_dim]
    tensor whose heads lie one after the other (a slice of a fused
    projection's rows is fine)."""
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.dim() != 3 or t.shape[2] != dim:
        raise ValueError(f"{name} must be [T, heads, {dim}]")
    if t.device != dev:
        raise ValueError(f"{name} must be on the cache's device (got {t.device})")
    if t.dtype != torch.bfloat16:
        raise TypeError(f"{name} must be {torch.bfloat16} (got {t.dtype})")
    T, heads, _ = t.shape
    if T and ((t.stride(2) != 1 and dim > 1) or (t.stride(1) != dim and heads > 1)):
        raise ValueError(f"{name}: the heads of a token must be contiguous")
    stride = t.stride(0) if T > 1 else max(heads * dim, 1)
    return t.data_ptr(), stride, T, heads


def _seqs_arg(block_table, seq_lens, cu_q, T: int, dev):
    if block_table.dim() != 2 or seq_lens.dim() != 1 or block_table.shape[0] != seq_lens.shape[0]:
        raise ValueError("block_table must be [B, width] and seq_lens [B]")
    B, width = block_table.shape
    if cu_q is None:
        if T != B:
            raise ValueError("without cu_q there is one new token for each sequence")
    elif tuple(cu_q.shape) != (B + 1,):
        raise ValueError("cu_q must be [B + 1]")
    return (_dev_ptr(block_table, "block_table", torch.int32, dev), width,
            _dev_ptr(seq_lens, "seq_lens", torch.int32, dev), _dev_ptr(cu_q, "cu_q", torch.int32, dev), B)


def _use_on(stream, dev, tensors) -> None:
    """Tell the allocator that a stream other than the current one uses these."""
    if stream is not None and stream != torch.cuda.current_stream(dev):
        for t in tensors:
            if isinstance(t, torch.Tensor):
                t.record_stream(stream)


def _empty(shape, dtype, dev, stream) -> torch.Tensor:
    """An output, allocated on the stream that the call runs on."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=dev)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=dev)


def kv_append(cache: dict, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
              cu_q: torch.Tensor | None = None, *, q: torch.Tensor | None = None, cos: torch.Tensor | None = None,
              sin: torch.Tensor | None = None, interleaved: bool = False, q_out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor | None:
    """Append the new tokens to the cache (``mhc_kv_append``).

    k, v bf16 [T, heads, head_dim]; q bf16 [T, q_heads, head_dim] or None.
    cos, sin fp32 [positions, rotary_dim / 2] or None (no rotation): keys and
    queries are rotated by their positions, in pairs (i, i + rotary_dim / 2)
    or, ``interleaved``, (2i, 2i + 1).  The cache is written in place; returns
    the rotated queries (``q_out``, which may be q itself), or None without q.
    """
    lib = load_library()
    c, dev = _cache_arg(cache)
    kp, ks, T, heads = _rows_arg(k, "k", c.head_dim, dev)
    vp, vs, Tv, hv = _rows_arg(v, "v", c.head_dim, dev)
    if (T, heads) != (Tv, hv) or heads != c.heads:
        raise ValueError("k and v must be [T, heads, head_dim] with the cache's heads")
    table = _seqs_arg(block_table, seq_lens, cu_q, T, dev)
    qa = (None, 0, 0, None, 0)
    if q is not None:
        qp, qs, Tq, hq = _rows_arg(q, "q", c.head_dim, dev)
        if Tq != T:
            raise ValueError("q must have as many tokens as k and v")
        if q_out is None:
            q_out = _empty((T, hq, c.head_dim), torch.bfloat16, dev, stream)
        op, os_, To, ho = _rows_arg(q_out, "q_out", c.head_dim, dev)
        if (To, ho) != (T, hq):
            raise ValueError("q_out must have q's shape")
        qa = (qp, qs, hq, op, os_)
    elif q_out is not None:
        raise ValueError("q_out without q")
    rows, dim = 0, 0
    if (cos is None) != (sin is None):
        raise ValueError("cos and sin go together")
    if cos is not None:
        if cos.dim() != 2 or cos.shape != sin.shape:
            raise ValueError("cos and sin must be [positions, rotary_dim / 2]")
        rows, dim = cos.shape[0], 2 * cos.shape[1]
    _use_on(stream, dev, (*cache.values(), k, v, q, q_out, cos, sin, block_table, seq_lens, cu_q))
    with torch.cuda.device(dev):
        st = lib.mhc_kv_append(c, kp, ks, vp, vs, *qa, _dev_ptr(cos, "cos", torch.float32, dev),
                               _dev_ptr(sin, "sin", torch.float32, dev), rows, dim, int(bool(interleaved)),
                               *table, T, _stream_ptr(stream, dev))
    _check("mhc_kv_append", st)
    return q_out


def kv_workspace_for(cache: dict, q_heads: int, B: int, T: int, stream=None) -> torch.Tensor | None:
    """A cached device workspace big enough for ``kv_attend`` (None when it
    needs none); one buffer for each (device, stream), as ``workspace_for``."""
    c, dev = _cache_arg(cache)
    return _workspace(c, dev, q_heads, B, T, stream)


def _workspace(c: _Cache, dev, q_heads: int, B: int, T: int, stream):
    di = _device_index(dev)
    with torch.cuda.device(di):
        need = int(load_library().mhc_kv_attend_workspace_bytes(c, q_heads, B, T))
        if need == 0:
            return None
        s = stream if stream is not None else torch.cuda.current_stream(di)
        key = ("kv", di, s.cuda_stream)
        buf = _workspaces.get(key)
        if buf is None or buf.numel() < need:
            with torch.cuda.stream(s):
                buf = torch.empty(need, dtype=torch.uint8, device=torch.device("cuda", di))
            _workspaces[key] = buf
    return buf


def kv_attend(q: torch.Tensor, cache: dict, block_table: torch.Tensor, seq_lens: torch.Tensor,
              cu_q: torch.Tensor | None = None, *, softmax_scale: float | None = None,
              out: torch.Tensor | None = None, lse: torch.Tensor | None = None, return_lse: bool = False,
              workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Causal attention of the new tokens over the cache (``mhc_kv_attend``).

    q bf16 [T, q_heads, head_dim], rotated; q_heads a multiple of the cache's
    heads.  softmax_scale defaults to head_dim ** -0.5.  Returns {"out": bf16
    [T, q_heads, head_dim][, "lse": fp32 [T, q_heads]]}; ``out`` and ``lse``
    may supply them.
    """
    lib = load_library()
    c, dev = _cache_arg(cache)
    qp, qs, T, heads = _rows_arg(q, "q", c.head_dim, dev)
    table = _seqs_arg(block_table, seq_lens, cu_q, T, dev)
    if out is None:
        out = _empty((T, heads, c.head_dim), torch.bfloat16, dev, stream)
    if lse is None and return_lse:
        lse = _empty((T, heads), torch.float32, dev, stream)
    if tuple(out.shape) != (T, heads, c.head_dim) or (lse is not None and tuple(lse.shape) != (T, heads)):
        raise ValueError("out / lse have the wrong shape")
    if softmax_scale is None:
        softmax_scale = 1.0 / math.sqrt(c.head_dim)
    if workspace is None:
        workspace = _workspace(c, dev, heads, table[-1], T, stream)
    ws, ws_bytes = (None, 0) if workspace is None else \
        (_dev_ptr(workspace, "workspace", torch.uint8, dev), workspace.numel())
    _use_on(stream, dev, (*cache.values(), q, out, lse, block_table, seq_lens, cu_q))
    with torch.cuda.device(dev):
        st = lib.mhc_kv_attend(c, qp, qs, heads, *table, T, float(softmax_scale),
                               _dev_ptr(out, "out", torch.bfloat16, dev), _dev_ptr(lse, "lse", torch.float32, dev),
                               ws, ws_bytes, _stream_ptr(stream, dev))
    _check("mhc_kv_attend", st)
    o = {"out": out}
    if lse is not None:
        o["lse"] = lse
    return o
