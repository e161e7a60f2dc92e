"""Reading part of the paged cache, for torch tensors: bounds of its pages, the
pages that they select for each query, and the attention over those and over
prefixes that sequences share.  The layouts, limits and device errors are
described in include/dspark.h."""
from __future__ import annotations

import math
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


class SparseWorkspace:
    """Device scratch for sparse_attention on this cache (or one of its sizes),
    for (B, T, heads) and lists of ``count`` pages or anything smaller in B, T and
    count."""

    def __init__(self, cache: PagedCache, B: int, T: int, heads: int, count: int):
        fn = "dspark_sparse_workspace_bytes"
        self.nbytes, self.buffer = _scratch(fn, cache, int(getattr(_lib.load(), fn)(cache._ref, B, T, heads, count)))


class PrefixWorkspace:
    """Device scratch for prefix_attention, sized for (B, T, heads, kv_heads,
    head_dim) or anything smaller in B and T."""

    def __init__(self, B: int, T: int, heads: int, kv_heads: int, head_dim: int, device=None):
        n = int(_lib.load().dspark_prefix_workspace_bytes(B, T, heads, kv_heads, head_dim))
        if n == 0:
            raise DsparkError("dspark_prefix_workspace_bytes", 2)
        self.nbytes = n
        self.buffer = torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def _attend(cache, fn, layer, q, length, special, make, mask, token_count, scale, seq, out, lse, with_lse,
            workspace, stream):
    """A call of the attentions below: ``special`` are the arguments between q
    and the mask."""
    B, T, heads, D = q.shape
    full = (B, T, heads, cache.head_dim)
    at = _ptr_of(cache, "q", q, cache.dtype, full)
    stride = 0
    if mask is not None and mask.dim() == 2:
        stride = T
    if out is None:
        with _on(stream):
            out = torch.empty_like(q)
    if lse is None and with_lse:
        with _on(stream):
            lse = torch.empty((B, T, heads), dtype=torch.float32, device=cache.device)
    workspace = _workspace(cache, workspace, stream, make)
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    i32, shape = torch.int32, (B,)
    _call(cache, fn, stream, layer, _ptr_of(cache, "seq", seq, i32, shape),
          _ptr_of(cache, "length", length, i32, shape),
          _ptr_of(cache, "token_count", token_count, i32, shape), at, *special,
          _ptr_of(cache, "mask", mask, torch.int64, (B, T) if stride else (T,)), stride, scale, B, T, heads,
          _ptr_of(cache, "out", out, cache.dtype, full),
          _ptr_of(cache, "lse", lse, torch.float32, (B, T, heads)), workspace.buffer.data_ptr(), workspace.nbytes)
    return out, lse


def sparse_attention(cache: PagedCache, layer: int, q, length, pages, *, mask=None, token_count=None,
                     scale: Optional[float] = None, seq=None, out=None, lse=None, with_lse: bool = False,
                     workspace: Optional[SparseWorkspace] = None, stream=None):
    """Attention of drafted tokens q [B, T, heads, D] over part of the cache of
    ``layer``: the full pages that ``pages`` [B, T, kv_heads, count] names (or
    [B, 1, kv_heads, count], for all tokens of a sequence alike; select_pages
    makes both), the committed tokens behind the last full page, and the drafted
    tokens that mask allows.  The other arguments and the results are those of
    tree_attention."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, heads, D]")
    if pages.dim() != 4:
        raise TypeError("pages must be int32 [B, T or 1, kv_heads, count]")
    B, T, heads, _ = q.shape
    lists, count = (1 if pages.shape[1] == 1 else T), pages.shape[3]
    special = (_ptr_of(cache, "pages", pages, torch.int32, (B, lists, cache.kv_heads, count)), count,
               1 if lists == 1 else 0)
    return _attend(cache, "dspark_sparse_attention", layer, q, length, special,
                   lambda: SparseWorkspace(cache, B, T, heads, count), mask, token_count, scale, seq, out, lse,
                   with_lse, workspace, stream)


def prefix_attention(cache: PagedCache, layer: int, q, length, group_start, prefix, *, mask=None,
                     token_count=None, scale: Optional[float] = None, seq=None, out=None, lse=None,
                     with_lse: bool = False, workspace: Optional[PrefixWorkspace] = None, stream=None):
    """tree_attention for sequences that share prefixes (cache_fork): rows
    group_start[g] .. group_start[g + 1] - 1 ([groups + 1] int32) share their
    first prefix[g] ([groups] int32) committed tokens, which are read once for
    all of them, through the pages of the first.  The other arguments and the
    results are those of tree_attention without a window."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, heads, D]")
    B, T, heads, D = q.shape
    i32, groups = torch.int32, _batch(prefix)
    special = (_ptr_of(cache, "group_start", group_start, i32, (groups + 1,)),
               _ptr_of(cache, "prefix", prefix, i32, (groups,)), groups)
    return _attend(cache, "dspark_prefix_attention", layer, q, length, special,
                   lambda: PrefixWorkspace(B, T, heads, cache.kv_heads, D, device=cache.device), mask, token_count,
                   scale, seq, out, lse, with_lse, workspace, stream)
