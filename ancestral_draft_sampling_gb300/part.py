"""Reading part of the paged cache, for torch tensors: bounds of its pages, and
the pages that they select for each query.  The layouts, limits and device
errors are described in include/dspark.h."""
from __future__ import annotations

from typing import Optional

import torch

from . import _lib
from ._lib import DsparkError
from .cache import PagedCache, _batch, _call, _on, _ptr_of


def _bounds_shape(cache: PagedCache):
    return (cache.layers, cache.num_pages, cache.kv_heads, 2, cache.head_dim)


def cache_bounds(cache: PagedCache, start, length, *, bounds=None, seq=None, stream=None):
    """The smallest and largest keys, in every layer, of the pages that the
    sequences have filled between ``start`` and ``length`` committed tokens
    ([B] int32 both).  Returns bounds [layers, num_pages, kv_heads, 2, head_dim]
    of the cache's dtype; a new one holds nothing of other pages."""
    i32, shape = torch.int32, (_batch(length),)
    at = _ptr_of(cache, "length", length, i32, shape)
    if bounds is None:
        with _on(stream):
            bounds = torch.zeros(_bounds_shape(cache), dtype=cache.dtype, device=cache.device)
    _call(cache, "dspark_cache_bounds", stream, _ptr_of(cache, "seq", seq, i32, shape),
          _ptr_of(cache, "start", start, i32, shape), at, shape[0],
          _ptr_of(cache, "bounds", bounds, cache.dtype, _bounds_shape(cache)))
    return bounds


def _scratch(fn, cache, nbytes):
    if nbytes == 0:
        raise DsparkError(fn, 2)
    return nbytes, torch.empty(nbytes, dtype=torch.uint8, device=cache.device)


class SelectWorkspace:
    """Device scratch for select_pages on this cache (or one of its sizes), for
    (B, T) or anything smaller; ``shared``: for shared lists only."""

    def __init__(self, cache: PagedCache, B: int, T: int, shared: bool = False):
        fn = "dspark_select_workspace_bytes"
        self.nbytes, self.buffer = _scratch(
            fn, cache, int(getattr(_lib.load(), fn)(cache._ref, B, T, 1 if shared else 0)))


def _workspace(cache, workspace, stream, make):
    if workspace is None:
        with _on(stream):
            return make()
    if workspace.buffer.get_device() != cache.index:
        raise ValueError("workspace must be on the cache's device")
    return workspace


def select_pages(cache: PagedCache, layer: int, bounds, q, length, count: int, *, first: int = 0,
                 last: int = 0, shared: bool = False, token_count=None, seq=None, pages=None,
                 workspace: Optional[SelectWorkspace] = None, stream=None):
    """For each drafted token of q [B, T, heads, D] and key head (``shared``: for
    all tokens of a sequence together) the ``count`` full pages whose ``bounds``
    (cache_bounds) allow the largest products with the queries, the sequence's
    ``first`` first and ``last`` last ones always among them.  Returns pages
    [B, T, kv_heads, count] ([B, 1, ...] if shared) int32: numbers within the
    sequence, ascending, -1 behind them; sparse_attention takes them."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, heads, D]")
    B, T, heads, _ = q.shape
    i32, shape = torch.int32, (B,)
    at = _ptr_of(cache, "q", q, cache.dtype, (B, T, heads, cache.head_dim))
    if pages is None:
        with _on(stream):
            pages = torch.full((B, 1 if shared else T, cache.kv_heads, count), -1, dtype=i32,
                               device=cache.device)
    workspace = _workspace(cache, workspace, stream, lambda: SelectWorkspace(cache, B, T, shared))
    _call(cache, "dspark_select_pages", stream, layer, _ptr_of(cache, "seq", seq, i32, shape),
          _ptr_of(cache, "length", length, i32, shape),
          _ptr_of(cache, "token_count", token_count, i32, shape), at,
          _ptr_of(cache, "bounds", bounds, cache.dtype, _bounds_shape(cache)), count, first, last,
          1 if shared else 0, B, T, heads,
          _ptr_of(cache, "pages", pages, i32, (B, 1 if shared else T, cache.kv_heads, count)),
          workspace.buffer.data_ptr(), workspace.nbytes)
    return pages
