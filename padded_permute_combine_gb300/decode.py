"""Python binding of include/moe_decode.h: what a decode step needs around the
few-token MoE layer (same names, same semantics).

As in ops.py this is argument marshalling only. A cache is a pair of tensors
[pages, page_size, kv_heads, head_dim] with any strides but in the last
dimension (tokens first, or heads first as a transposed view), the same for keys
and values. The plain call (right arguments, outputs to be allocated) is
marshalled by csrc/decode_calls.cpp; it answers None to any other, which is then
taken step by step here, with a message for what is wrong. The small outputs that
a plain call allocates share one allocation, which lives as long as any of them
(a page table kept from moe_cache_compact holds src and dst too): pass ``out``, or
clone what is kept for long, where that matters.

Nothing here is differentiable: outputs never require gradients, whatever the
inputs do, and caches are written in place behind autograd's back.
"""
from __future__ import annotations

import ctypes
from typing import NamedTuple, Sequence

import torch

from . import _lib
from .block import _done, _on, _status, _stream, _take, _workspace
from .ops import _act_dtype, _need

_I32 = torch.int32


class CacheFork(NamedTuple):
    page_table: torch.Tensor  # [rows, width] int32
    lengths: torch.Tensor     # [rows] int32
    src: torch.Tensor         # [rows] int32: page that row r copies, or -1
    dst: torch.Tensor         # [rows] int32: where to


class CacheCompact(NamedTuple):
    page_table: torch.Tensor  # [rows, width] int32
    src: torch.Tensor         # [num_pages // 2] int32: pages that move, then -1
    dst: torch.Tensor         # [num_pages // 2] int32: where to
    count: torch.Tensor       # [1] int32: how many


def _tensor(t, name: str, dims: int, dtype: torch.dtype | None, device) -> torch.Tensor:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda:
        raise ValueError("%s must be a CUDA tensor" % name)
    if t.dim() != dims:
        raise ValueError("%s must be %d-D, got %s" % (name, dims, list(t.shape)))
    if dtype is not None and t.dtype != dtype:
        raise TypeError("%s must be %s, got %s" % (name, dtype, t.dtype))
    if device is not None and t.device != device:
        raise ValueError("%s is on %s, expected %s" % (name, t.device, device))
    return t


def _int(v: int, name: str, bits: int = 32) -> int:
    if not -2 ** (bits - 1) <= v < 2 ** (bits - 1):  # ctypes would cut it
        raise ValueError("%s does not fit %d bits: %d" % (name, bits, v))
    return v


def _strides(t: torch.Tensor, name: str, apart: bool) -> tuple:
    """The strides of a tensor that is contiguous in its last dimension (0 for
    dimensions of one element). ``apart``: elements may not overlap."""
    if t.shape[-1] > 1 and t.stride(-1) != 1:
        raise ValueError("%s must be contiguous in its last dimension" % name)
    s = tuple(0 if n <= 1 else d for n, d in zip(t.shape[:-1], t.stride()[:-1]))
    if apart and t.numel():
        reach = t.shape[-1]
        for d, n in sorted((d, n) for d, n in zip(s, t.shape[:-1]) if n > 1):
            if d < reach:
                raise ValueError("%s must not overlap itself" % name)
            reach += d * (n - 1)
    return s


def _cache(k_cache, v_cache, device=None) -> _lib.KvCache:
    _tensor(k_cache, "k_cache", 4, None, device)
    dt = _act_dtype(k_cache, "k_cache")
    _tensor(v_cache, "v_cache", 4, k_cache.dtype, k_cache.device)
    if v_cache.shape != k_cache.shape:
        raise ValueError("v_cache must be %s, got %s" % (list(k_cache.shape), list(v_cache.shape)))
    s = _strides(k_cache, "k_cache", True)
    if _strides(v_cache, "v_cache", True) != s:
        raise ValueError("k_cache and v_cache must have the same strides")
    n, *rest = k_cache.shape
    page, heads, dim = (_int(v, "k_cache's %s" % name) for v, name in zip(rest, ("page size", "kv heads", "head size")))
    return _lib.KvCache(k_cache.data_ptr() or None, v_cache.data_ptr() or None, n, *s, dt, page, heads, dim)


def _heads(t, name: str, rows: int, heads: int | None, like: torch.Tensor) -> _lib.Heads:
    _tensor(t, name, 3, like.dtype, like.device)
    want = (rows, t.shape[1] if heads is None else heads, like.shape[3])
    if t.shape != want:
        raise ValueError("%s must be %s, got %s" % (name, list(want), list(t.shape)))
    return _lib.Heads(t.data_ptr() or None, *_strides(t, name, False))


def _table(page_table, lengths, device) -> tuple[int, int, int, int, int]:
    """Address, row stride and width of the table, rows, and the lengths' address."""
    _tensor(page_table, "page_table", 2, _I32, device)
    rows, width = page_table.shape
    stride, = _strides(page_table, "page_table", False)
    if rows > 1 and stride < width:
        raise ValueError("page_table must have rows that do not overlap")
    return page_table.data_ptr() or None, stride, width, rows, _take(lengths, (rows,), _I32, "lengths", device) or None


def attention_workspace(num_seqs: int, num_heads: int, num_kv_heads: int, head_dim: int, device) -> torch.Tensor:
    """Workspace of moe_attention_decode (one per stream that may run it at the same time)."""
    with _on(torch.device(device)):
        size = _lib.load().moe_attention_decode_workspace_size(num_seqs, num_heads, num_kv_heads, head_dim)
    return torch.empty(size, dtype=torch.uint8, device=device)


def moe_attention_decode(q: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor, page_table: torch.Tensor,
                         lengths: torch.Tensor, k_new: torch.Tensor | None = None, v_new: torch.Tensor | None = None,
                         scale: float | None = None, window: int = 0, out: torch.Tensor | None = None,
                         lse: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
                         status: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor]:
    """Attention of one new token of every sequence over its cache:
    q [B, heads, head_dim], k_cache and v_cache [pages, page_size, kv_heads,
    head_dim], page_table [B, width] int32, lengths [B] int32 (the new token
    counted) -> (out [B, heads, head_dim], lse [B, heads] fp32). k_new and v_new
    [B, kv_heads, head_dim] are written to position lengths - 1 on the way; a
    token whose length lies beyond the table (a fork without a column to grow
    into), or whose page is bad, is left out, and ``status`` says so.
    scale: head_dim ** -0.5 by default; window: the last positions that are
    looked at, 0 for all."""
    if out is None and lse is None and workspace is None and status is None:
        done = (_lib.calls or _lib.load_calls()).attention_decode(
            q, k_cache, v_cache, page_table, lengths, k_new, v_new, scale, window)
        if done is not None:
            return done
    _tensor(q, "q", 3, None, None)
    dev = q.device
    cache = _cache(k_cache, v_cache, dev)
    B, H, D = q.shape
    _int(H, "q's heads")
    _int(window, "window", 64)
    q_at = _heads(q, "q", B, None, k_cache)
    table, stride, width, rows, lengths_at = _table(page_table, lengths, dev)
    if rows != B:
        raise ValueError("page_table must have %d rows, has %d" % (B, rows))
    if (k_new is None) != (v_new is None):
        raise ValueError("k_new and v_new go together")
    new = [None if t is None else ctypes.byref(_heads(t, name, B, cache.num_kv_heads, k_cache))
           for t, name in ((k_new, "k_new"), (v_new, "v_new"))]
    if out is None:
        out = torch.empty((B, H, D), dtype=q.dtype, device=dev)
    if lse is None:
        lse = torch.empty((B, H), dtype=torch.float32, device=dev)
    out_at, lse_at = _take(out, (B, H, D), q.dtype, "out", dev), _take(lse, (B, H), torch.float32, "lse", dev)
    lib = _lib.load()
    with _on(dev):
        ws = _workspace(workspace, lib.moe_attention_decode_workspace_size(B, H, cache.num_kv_heads, D), dev)
        rc = lib.moe_attention_decode(
            ctypes.byref(cache), ctypes.byref(q_at), H, table, stride, width, lengths_at, B, *new,
            D ** -0.5 if scale is None else scale, window, out_at, lse_at, ws.data_ptr(), ws.numel(), _status(status, dev),
            _stream(dev))
    _done("moe_attention_decode", rc)
    return out, lse


def moe_cache_write(k: torch.Tensor, v: torch.Tensor, k_cache: torch.Tensor, v_cache: torch.Tensor,
                    page_table: torch.Tensor, offsets: torch.Tensor, lengths: torch.Tensor,
                    status: torch.Tensor | None = None) -> None:
    """Writes the keys and values of many tokens into the cache: rows
    offsets[b] .. offsets[b + 1] - 1 of k and v [tokens, kv_heads, head_dim] are
    the last tokens of sequence b, whose length with them is lengths[b]."""
    if status is None and (_lib.calls or _lib.load_calls()).cache_write(
            k, v, k_cache, v_cache, page_table, offsets, lengths) is not None:
        return
    cache = _cache(k_cache, v_cache)
    dev = k_cache.device
    _tensor(k, "k", 3, None, None)
    T = k.shape[0]
    k_at, v_at = _heads(k, "k", T, cache.num_kv_heads, k_cache), _heads(v, "v", T, cache.num_kv_heads, k_cache)
    table, stride, width, rows, lengths_at = _table(page_table, lengths, dev)
    offsets_at = _take(offsets, (rows + 1,), _I32, "offsets", dev)
    with _on(dev):
        rc = _lib.load().moe_cache_write(
            ctypes.byref(cache), ctypes.byref(k_at), ctypes.byref(v_at), T, offsets_at, table, stride, width, lengths_at, rows,
            _status(status, dev), _stream(dev))
    _done("moe_cache_write", rc)


def moe_cache_fork(page_table: torch.Tensor, lengths: torch.Tensor, parents: torch.Tensor, page_size: int, num_pages: int,
                   grow: int = 1, width: int | None = None, out: CacheFork | None = None,
                   status: torch.Tensor | None = None) -> CacheFork:
    """The page table of the next step: row r goes on from row parents[r] (-1:
    an empty row) with room for ``grow`` more tokens; see include/moe_decode.h.
    The copies src -> dst are moe_cache_copy's to make. ``width``: columns of the
    new table, page_table's by default."""
    if out is None and status is None:
        done = (_lib.calls or _lib.load_calls()).cache_fork(page_table, lengths, parents, page_size, num_pages, grow, width)
        if done is not None:
            return tuple.__new__(CacheFork, done)
    _tensor(page_table, "page_table", 2, _I32, None)
    dev = page_table.device
    table, stride, old, rows, lengths_at = _table(page_table, lengths, dev)
    for v, name, bits in ((page_size, "page_size", 32), (num_pages, "num_pages", 64), (grow, "grow", 64)):
        _int(v, name, bits)
    _tensor(parents, "parents", 1, _I32, dev)
    R = parents.shape[0]
    parents_at = _take(parents, (R,), _I32, "parents", dev)
    if out is None:
        new = lambda *shape: torch.empty(shape, dtype=_I32, device=dev)  # noqa: E731
        out = CacheFork(new(R, old if width is None else width), new(R), new(R), new(R))
    new_width = out[0].shape[1] if width is None else width
    at = [_take(t, shape, _I32, name, dev) or None for t, shape, name in
          zip(out, ((R, new_width), (R,), (R,), (R,)), ("out.page_table", "out.lengths", "out.src", "out.dst"))]
    with _on(dev):
        rc = _lib.load().moe_cache_fork(
            table, stride, old, lengths_at, rows, parents_at or None, R, page_size, num_pages, grow, at[0], new_width, *at[1:],
            _status(status, dev), _stream(dev))
    _done("moe_cache_fork", rc)
    return CacheFork(*out)


def moe_cache_compact(page_table: torch.Tensor, lengths: torch.Tensor, page_size: int, num_pages: int,
                      out: CacheCompact | None = None, status: torch.Tensor | None = None) -> CacheCompact:
    """Moves the pages in use to the front of the pool: the table with the new
    numbers, and the copies src -> dst (``count`` of them) for moe_cache_copy."""
    if out is None and status is None:
        done = (_lib.calls or _lib.load_calls()).cache_compact(page_table, lengths, page_size, num_pages)
        if done is not None:
            return tuple.__new__(CacheCompact, done)
    _tensor(page_table, "page_table", 2, _I32, None)
    dev = page_table.device
    table, stride, width, rows, lengths_at = _table(page_table, lengths, dev)
    _int(page_size, "page_size")
    half = max(0, _int(num_pages, "num_pages", 64)) // 2
    if out is None:
        new = lambda *shape: torch.empty(shape, dtype=_I32, device=dev)  # noqa: E731
        out = CacheCompact(new(rows, width), new(half), new(half), new(1))
    at = [_take(t, shape, _I32, name, dev) or None for t, shape, name in
          zip(out, ((rows, width), (half,), (half,), (1,)), ("out.page_table", "out.src", "out.dst", "out.count"))]
    with _on(dev):
        rc = _lib.load().moe_cache_compact(
            table, stride, width, lengths_at, rows, page_size, num_pages, *at, _status(status, dev), _stream(dev))
    _done("moe_cache_compact", rc)
    return CacheCompact(*out)


def _pages(t, name: str, num_pages: int, device) -> _lib.CachePages:
    if not isinstance(t, torch.Tensor):
        raise TypeError("%s must be a torch.Tensor" % name)
    if not t.is_cuda or t.device != device:
        raise ValueError("%s must be on %s" % (name, device))
    if t.dim() < 1 or t.shape[0] != num_pages:
        raise ValueError("%s must have %d pages, got %s" % (name, num_pages, list(t.shape)))
    size = 1
    for d, n in sorted((d, n) for d, n in zip(t.stride()[1:], t.shape[1:]) if n != 1):
        if d != size and n > 0:
            raise ValueError("a page of %s must be one block of memory" % name)
        size *= n
    stride = t.stride(0) if num_pages > 1 else size
    if stride < size:
        raise ValueError("%s must have pages that do not overlap" % name)
    return _lib.CachePages(t.data_ptr() or None, stride * t.element_size(), size * t.element_size())


def moe_cache_copy(caches: Sequence[torch.Tensor], src: torch.Tensor, dst: torch.Tensor, count: torch.Tensor | None = None,
                   status: torch.Tensor | None = None) -> None:
    """Copies page src[i] to page dst[i] in every one of the caches ([pages,
    ...] of any type and any order of the dimensions behind the first, a page
    being one block of memory), in place. Pairs with -1 are passed over;
    ``count``: how many pairs there are (int32 [1] on the device)."""
    caches = list(caches)
    if status is None and (_lib.calls or _lib.load_calls()).cache_copy(caches, src, dst, count) is not None:
        return
    _need(src, _I32, "src")
    dev = src.device
    n = src.numel()
    src_at, dst_at = _take(src, (n,), _I32, "src", dev), _take(dst, (n,), _I32, "dst", dev)
    count_at = None if count is None else _take(count, (1,), _I32, "count", dev)
    num_pages = caches[0].shape[0] if caches and isinstance(caches[0], torch.Tensor) and caches[0].dim() else 0
    most = _lib.MOE_CACHE_MAX_CACHES
    entries = [_pages(t, "caches[%d]" % i, num_pages, dev) for i, t in enumerate(caches)]
    with _on(dev):
        for i in range(0, len(entries), most):
            some = (_lib.CachePages * len(entries[i:i + most]))(*entries[i:i + most])
            rc = _lib.load().moe_cache_copy(
                some, len(some), num_pages, src_at or None, dst_at or None, n, count_at, _status(status, dev), _stream(dev))
            _done("moe_cache_copy", rc)


def moe_beam_select(logits: torch.Tensor, scores: torch.Tensor, num_out: int, ended: torch.Tensor | None = None,
                    end_token: int = -1, out: tuple[torch.Tensor, torch.Tensor, torch.Tensor] | None = None,
                    workspace: torch.Tensor | None = None) -> tuple[torch.Tensor, torch.Tensor, torch.Tensor]:
    """Beam search's selection: logits [B, beams, vocab] and scores [B, beams]
    fp32 -> the num_out best of scores + log_softmax(logits) of each request,
    best first: (scores fp32, parents int32 = b * beams + beam, tokens int32),
    each [B, num_out]. A beam with ``ended`` (bool or uint8 [B, beams]) goes on
    with end_token alone, at the score that it has."""
    if out is None and workspace is None:
        done = (_lib.calls or _lib.load_calls()).beam_select(logits, scores, num_out, ended, end_token)
        if done is not None:
            return done
    _tensor(logits, "logits", 3, None, None)
    dt = _act_dtype(logits, "logits")
    dev = logits.device
    B, W, V = logits.shape
    for v, name in ((W, "beams"), (num_out, "num_out"), (end_token, "end_token")):
        _int(v, name)
    per_request, stride = _strides(logits, "logits", False)
    if W == 1:
        stride = per_request
    elif B > 1 and per_request != W * stride:
        raise ValueError("the rows of logits must be evenly spaced")
    if B * W > 1 and stride < V:
        raise ValueError("logits must have rows that do not overlap")
    scores_at = _take(scores, (B, W), torch.float32, "scores", dev)
    ended_at = None
    if ended is not None:
        if not isinstance(ended, torch.Tensor):
            raise TypeError("ended must be a torch.Tensor")
        ended_at = _take(ended, (B, W), torch.bool if ended.dtype == torch.bool else torch.uint8, "ended", dev)
    if out is None:
        out = (torch.empty((B, num_out), dtype=torch.float32, device=dev),
               *(torch.empty((B, num_out), dtype=_I32, device=dev) for _ in range(2)))
    at = [_take(t, (B, num_out), d, n, dev) or None for t, d, n in
          zip(out, (torch.float32, _I32, _I32), ("out[0]", "out[1]", "out[2]"))]
    lib = _lib.load()
    ws = _workspace(workspace, lib.moe_beam_select_workspace_size(B, W, V), dev)
    with _on(dev):
        rc = lib.moe_beam_select(
            logits.data_ptr() or None, dt, stride, scores_at or None, ended_at or None, B, W, V, num_out, end_token, *at,
            ws.data_ptr() or None, ws.numel(), _stream(dev))
    _done("moe_beam_select", rc)
    return tuple(out)
