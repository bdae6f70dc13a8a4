"""Paged 8-bit key/value cache: the calls of ``include/mhc_kv.h``.

    kv_cache(num_pages, heads, page_tokens, head_dim) -> dict
    kv_append(cache, k, v, block_table, seq_lens, cu_q=None, q=None, cos=None, sin=None, ...) -> Tensor | None
    kv_attend(q, cache, block_table, seq_lens, cu_q=None, ...) -> dict
    kv_fork(caches, block_table, seq_lens, parents=None, ...) -> dict
    kv_compact(caches, block_table, seq_lens, ...) -> dict

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

__all__ = ["kv_cache", "kv_append", "kv_attend", "kv_fork", "kv_compact", "kv_workspace_for"]

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
    lib.mhc_kv_append_norm.argtypes = [C, P, I64, P, I64, P, I64, I, P, I64, P, I64, P, I64, F, P, P, I64, I, I, P, I64, P,
                                       P, I64, I64, P]
    lib.mhc_kv_append_norm.restype = I
    lib.mhc_kv_attend.argtypes = [C, P, I64, I, P, I64, P, P, I64, I64, F, P, P, P, ctypes.c_size_t, P]
    lib.mhc_kv_attend.restype = I
    lib.mhc_kv_attend_window.argtypes = [C, P, I64, I, P, I64, P, P, I64, I64, F, I64, I64, P, P, P, ctypes.c_size_t, P]
    lib.mhc_kv_attend_window.restype = I
    lib.mhc_kv_fork.argtypes = [C, I, P, I64, P, I64, P, I64, P, I64, P, I64, I64, P, P, P, ctypes.c_size_t, P]
    lib.mhc_kv_fork.restype = I
    lib.mhc_kv_compact.argtypes = [C, I, P, I64, P, I64, P, P, P, P, ctypes.c_size_t, P]
    lib.mhc_kv_compact.restype = I
    lib.mhc_kv_fork_workspace_bytes.argtypes = [I64, I64, I64]
    lib.mhc_kv_fork_workspace_bytes.restype = ctypes.c_size_t
    lib.mhc_kv_compact_workspace_bytes.argtypes = [I64, I64]
    lib.mhc_kv_compact_workspace_bytes.restype = ctypes.c_size_t
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
              q_norm: torch.Tensor | None = None, k_norm: torch.Tensor | None = None, norm_eps: float = 1e-6,
              stream=None) -> torch.Tensor | None:
    """Append the new tokens to the cache (``mhc_kv_append``, ``mhc_kv_append_norm``).

    k, v bf16 [T, heads, head_dim]; q bf16 [T, q_heads, head_dim] or None;
    each may be a slice of a fused projection's rows.  cos, sin fp32
    [positions, rotary_dim / 2] or None (no rotation): keys and queries are
    rotated by their positions, in pairs (i, i + rotary_dim / 2) or,
    ``interleaved``, (2i, 2i + 1).  q_norm, k_norm bf16 [head_dim] or [heads,
    head_dim]: queries or keys are divided by their head's root mean square
    (``norm_eps`` is added to the mean) and multiplied by these weights before
    the rotation.  The cache is written in place; returns the rotated queries (``q_out``, which may be q itself), or None without q.
    """
    if stream is not None:
        with _on(stream, cache, (*cache.values(), k, v, q, q_out, cos, sin, block_table, seq_lens, cu_q, q_norm, k_norm)):
            return kv_append(cache, k, v, block_table, seq_lens, cu_q, q=q, cos=cos, sin=sin, interleaved=interleaved,
                             q_out=q_out, q_norm=q_norm, k_norm=k_norm, norm_eps=norm_eps)
    return (_module or _load()).append(cache["k"], cache["v"], cache["k_scale"], cache["v_scale"], k, v, block_table,
                                       seq_lens, cu_q, q, cos, sin, interleaved, q_out, q_norm, k_norm, norm_eps)


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
              window: int | None = None, sinks: int = 0, out: torch.Tensor | None = None,
              lse: torch.Tensor | None = None, return_lse: bool = False, workspace: torch.Tensor | None = None,
              stream=None) -> dict:
    """Causal attention of the new tokens over the cache (``mhc_kv_attend``, ``mhc_kv_attend_window``).

    q bf16 [T, q_heads, head_dim], rotated; q_heads a multiple of the cache's
    heads.  softmax_scale defaults to head_dim ** -0.5.  With a ``window`` a
    token sees the last ``window`` keys up to its own, and the sequence's first
    ``sinks``; pages of which no new token sees a key need not be there (-1 in
    the table).  Returns {"out": bf16 [T, q_heads, head_dim][, "lse": fp32 [T,
    q_heads]]}; ``out`` and ``lse`` may supply them.
    """
    if stream is not None:
        with _on(stream, cache, (*cache.values(), q, out, lse, block_table, seq_lens, cu_q, workspace)):
            return kv_attend(q, cache, block_table, seq_lens, cu_q, softmax_scale=softmax_scale, window=window,
                             sinks=sinks, out=out, lse=lse, return_lse=return_lse, workspace=workspace)
    out, lse = (_module or _load()).attend(q, cache["k"], cache["v"], cache["k_scale"], cache["v_scale"], block_table,
                                           seq_lens, cu_q, softmax_scale, out, lse, return_lse, workspace, window,
                                           sinks)
    return {"out": out} if lse is None else {"out": out, "lse": lse}


def _layers(caches, out, tensors, stream):
    """``_on`` for the calls that take all layers' caches."""
    if not caches or not all(isinstance(c, dict) for c in caches):
        raise ValueError("caches must be a cache or a sequence of caches")
    every = [t for c in caches for t in c.values()] + list((out or {}).values())
    return _on(stream, caches[0], (*every, *tensors))


def kv_fork(caches, block_table: torch.Tensor, seq_lens: torch.Tensor, parents: torch.Tensor | None = None, *,
            room=0, window: int | None = None, sinks: int = 0, held: torch.Tensor | None = None,
            out: dict | None = None, workspace: torch.Tensor | None = None, stream=None) -> dict:
    """The tables of the next step (``mhc_kv_fork``): place b goes on with place parents[b]'s tokens.

    caches: a cache, or the caches of all layers, which share page numbers.
    parents int32 [B], -1 for a place without tokens, or None (every place goes
    on with itself).  Full pages are shared, a part-filled one is copied but
    for the first place that goes on with it.  room: how many further tokens a
    place gets pages for, a number or int32 [B].  With a ``window`` (and
    ``sinks``) pages that no later token sees are let go.  held: bool
    [num_pages], pages that others go on using.  Every other page is free, and
    handed out from the lowest number on.  Returns {"block_table": int32 [B,
    width], "seq_lens": int32 [B]}, the lengths without the room; ``out`` may
    supply them (without parents they may be the call's own).
    ``device_status()`` is 6 where free pages ran out; the entries are -1 then.
    """
    caches = (caches,) if isinstance(caches, dict) else tuple(caches)
    if stream is not None:
        with _layers(caches, out, (block_table, seq_lens, parents, room, held, workspace), stream):
            return kv_fork(caches, block_table, seq_lens, parents, room=room, window=window, sinks=sinks, held=held,
                           out=out, workspace=workspace)
    o = out or {}
    table, lens = (_module or _load()).fork(caches, block_table, seq_lens, parents, room, window, sinks, held,
                                            o.get("block_table"), o.get("seq_lens"), workspace)
    return {"block_table": table, "seq_lens": lens}


def kv_compact(caches, block_table: torch.Tensor, seq_lens: torch.Tensor, *, held: torch.Tensor | None = None,
               out: dict | None = None, workspace: torch.Tensor | None = None, stream=None) -> dict:
    """Move the pages in use to the lowest numbers (``mhc_kv_compact``).

    caches, held as in ``kv_fork``; held pages stay where they are.  Returns
    {"block_table": int32 [B, width], the tables with the pages' new numbers,
    "pages": int32 [], how many pages, from the first on, hold all that are in
    use or held}; ``out`` may supply them (its table may be block_table itself).
    """
    caches = (caches,) if isinstance(caches, dict) else tuple(caches)
    if stream is not None:
        with _layers(caches, out, (block_table, seq_lens, held, workspace), stream):
            return kv_compact(caches, block_table, seq_lens, held=held, out=out, workspace=workspace)
    o = out or {}
    table, pages = (_module or _load()).compact(caches, block_table, seq_lens, held, o.get("block_table"),
                                                o.get("pages"), workspace)
    return {"block_table": table, "pages": pages}
