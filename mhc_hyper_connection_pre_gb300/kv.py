"""Paged 8-bit key/value cache: the calls of ``include/mhc_kv.h``.

    kv_cache(num_pages, heads, page_tokens, head_dim) -> dict
    kv_append(cache, k, v, block_table, seq_lens, cu_q=None, q=None, cos=None, sin=None, ...) -> Tensor | None
    kv_attend(q, cache, block_table, seq_lens, cu_q=None, ...) -> dict

A cache is a dict of tensors: "k", "v" float8_e4m3fn [num_pages, heads,
page_tokens, head_dim] and "k_scale", "v_scale" fp32 [num_pages, heads].
block_table int32 [B, width] holds each sequence's pages, seq_lens int32 [B]
each sequence's length with its new tokens, cu_q int32 [B + 1] where each
sequence's new tokens begin (None: one for each sequence).  The calls are
asynchronous; a bad index on the device is reported by ``device_status()``.

The tensors are checked and the outputs allocated in ``csrc/kv_binding.cpp``.
"""
from __future__ import annotations

import ctypes
import importlib.machinery
import importlib.util
import os
import threading

import torch

from . import MhcError, library_path, load_library

__all__ = ["kv_cache", "kv_append", "kv_attend", "kv_workspace_for"]

_lock = threading.Lock()
_module = None


class _Cache(ctypes.Structure):
    """mhc_kv_cache."""
    _fields_ = [("k", ctypes.c_void_p), ("v", ctypes.c_void_p), ("k_scale", ctypes.c_void_p),
                ("v_scale", ctypes.c_void_p), ("num_pages", ctypes.c_int64), ("heads", ctypes.c_int),
                ("page_tokens", ctypes.c_int), ("head_dim", ctypes.c_int)]


def declare(lib) -> None:
    """Argument types of the C entry points (called once by ``load_library``)."""
    P, I64, I, F = ctypes.c_void_p, ctypes.c_int64, ctypes.c_int, ctypes.c_float
    C = ctypes.POINTER(_Cache)
    lib.mhc_kv_append.argtypes = [C, P, I64, P, I64, P, I64, I, P, I64, P, P, I64, I, I, P, I64, P, P, I64, I64, P]
    lib.mhc_kv_append.restype = I
    lib.mhc_kv_attend.argtypes = [C, P, I64, I, P, I64, P, P, I64, I64, F, P, P, P, ctypes.c_size_t, P]
    lib.mhc_kv_attend.restype = I
    lib.mhc_kv_attend_workspace_bytes.argtypes = [C, I, I64, I64]
    lib.mhc_kv_attend_workspace_bytes.restype = ctypes.c_size_t


def _load():
    """Load _mhc_kv.so (built by ``build.py``); raises if it is absent."""
    global _module
    with _lock:
        if _module is None:
            load_library()
            path = os.path.join(os.path.dirname(library_path()), "_mhc_kv.so")
            if not os.path.exists(path):
                raise RuntimeError(f"_mhc_kv.so not found at {path}: build it with "
                                   "`python -m mhc_hyper_connection_pre_gb300.build` (no fallback exists)")
            loader = importlib.machinery.ExtensionFileLoader("_mhc_kv", path)
            m = importlib.util.module_from_spec(importlib.util.spec_from_file_location("_mhc_kv", path, loader=loader))
            loader.exec_module(m)
            m.set_error(MhcError)
            _module = m
        return _module


def captured_workspace(user: int, need: int, device: int, stream) -> torch.Tensor | None:
    """The workspace of the capture under way on ``stream``, which its graph keeps alive; None if there is none."""
    return (_module or _load()).captured(user, need, device, stream.cuda_stream)


def kv_cache(num_pages: int, heads: int, page_tokens: int = 64, head_dim: int = 128, *, device="cuda") -> dict:
    """An empty cache of one layer (every code and scale zero)."""
    shape = (num_pages, heads, page_tokens, head_dim)
    return {"k": torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
            "v": torch.zeros(shape, dtype=torch.uint8, device=device).view(torch.float8_e4m3fn),
            "k_scale": torch.zeros(num_pages, heads, dtype=torch.float32, device=device),
            "v_scale": torch.zeros(num_pages, heads, dtype=torch.float32, device=device)}


def _on(stream, cache, tensors=()):
    """A context in which ``stream``, of the cache's device, is the current
    stream, and so allocates the outputs; the allocator learns that it uses
    ``tensors``."""
    if isinstance(cache["k"], torch.Tensor) and cache["k"].device != stream.device:
        raise ValueError(f"stream must be on the cache's device {cache['k'].device} (got {stream.device})")
    for t in tensors:
        if isinstance(t, torch.Tensor) and t.is_cuda:
            t.record_stream(stream)
    return torch.cuda.stream(stream)


def kv_append(cache: dict, k: torch.Tensor, v: torch.Tensor, block_table: torch.Tensor, seq_lens: torch.Tensor,
              cu_q: torch.Tensor | None = None, *, q: torch.Tensor | None = None, cos: torch.Tensor | None = None,
              sin: torch.Tensor | None = None, interleaved: bool = False, q_out: torch.Tensor | None = None,
              stream=None) -> torch.Tensor | None:
    """Append the new tokens to the cache (``mhc_kv_append``).

    k, v bf16 [T, heads, head_dim]; q bf16 [T, q_heads, head_dim] or None;
    each may be a slice of a fused projection's rows.  cos, sin fp32
    [positions, rotary_dim / 2] or None (no rotation): keys and queries are
    rotated by their positions, in pairs (i, i + rotary_dim / 2) or,
    ``interleaved``, (2i, 2i + 1).  The cache is written in place; returns the
    rotated queries (``q_out``, which may be q itself), or None without q.
    """
    if stream is not None:
        with _on(stream, cache, (*cache.values(), k, v, q, q_out, cos, sin, block_table, seq_lens, cu_q)):
            return kv_append(cache, k, v, block_table, seq_lens, cu_q, q=q, cos=cos, sin=sin, interleaved=interleaved,
                             q_out=q_out)
    return (_module or _load()).append(cache["k"], cache["v"], cache["k_scale"], cache["v_scale"], k, v, block_table,
                                       seq_lens, cu_q, q, cos, sin, interleaved, q_out)


def kv_workspace_for(cache: dict, q_heads: int, B: int, T: int, stream=None) -> torch.Tensor | None:
    """The device workspace that ``kv_attend`` uses when it is given none
    (None when it needs none): one buffer for each (device, stream), grown on
    demand and allocated on that stream, as ``workspace_for``.  A graph has
    one of its own: while the stream is being captured this is the capture's,
    which lives as long as the graph.  Passed on as ``workspace`` to calls on
    another stream or in a graph, a buffer is shared with this stream's own
    calls, and kept alive by whoever holds it."""
    if stream is not None:
        with _on(stream, cache):
            return kv_workspace_for(cache, q_heads, B, T)
    return (_module or _load()).workspace(cache["k"], cache["v"], cache["k_scale"], cache["v_scale"], q_heads, B, T)


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
    if stream is not None:
        with _on(stream, cache, (*cache.values(), q, out, lse, block_table, seq_lens, cu_q, workspace)):
            return kv_attend(q, cache, block_table, seq_lens, cu_q, softmax_scale=softmax_scale, out=out, lse=lse,
                             return_lse=return_lse, workspace=workspace)
    out, lse = (_module or _load()).attend(q, cache["k"], cache["v"], cache["k_scale"], cache["v_scale"], block_table,
                                           seq_lens, cu_q, softmax_scale, out, lse, return_lse, workspace)
    return {"out": out} if lse is None else {"out": out, "lse": lse}
