"""The paged key/value cache and the attention of drafted tokens over it, for
torch tensors: checks of dtypes, shapes and devices, and raw pointers to the
library.  The layouts, limits and device errors are described in
include/dspark.h."""
from __future__ import annotations

import ctypes
import math
from typing import Optional

from . import _lib
from ._lib import BF16, F32, DsparkError

CONTROL_WORDS = 64 + 2 * 1024  # DSPARK_CACHE_CONTROL_WORDS


def _torch():
    import torch
    return torch


def _ptr(t) -> Optional[int]:
    return None if t is None else t.data_ptr()


class PagedCache:
    """A paged key/value cache: ``pool`` [layers, 2, num_pages, kv_heads,
    page_size, head_dim], float32 or bfloat16, and the tables that say which
    sequence holds which page.  A new cache is empty: cache_reserve gives its
    sequences pages.  The lengths of the sequences are the caller's."""

    def __init__(self, layers: int, num_pages: int, page_size: int, kv_heads: int,
                 head_dim: int, max_seqs: int, max_pages: int, dtype=None,
                 device=None, stream=None):
        torch = _torch()
        device = device or "cuda"
        i32 = dict(dtype=torch.int32, device=device)
        self._set(torch.empty(layers, 2, num_pages, kv_heads, page_size, head_dim,
                              dtype=dtype or torch.bfloat16, device=device),
                  torch.empty(max_seqs, max_pages, **i32), torch.empty(max_seqs, **i32),
                  torch.empty(num_pages, **i32), torch.empty(num_pages, **i32),
                  torch.empty(CONTROL_WORDS, **i32))
        with self._current():
            _check("dspark_cache_init", _lib.load().dspark_cache_init(
                self._ref, self._stream(stream)))

    @classmethod
    def from_tensors(cls, pool, block_table, page_count, ref_count, free_list, control):
        """A cache over tensors that the caller has made and filled: pool,
        block_table [max_seqs, max_pages], page_count [max_seqs], ref_count
        and free_list [num_pages], control [CONTROL_WORDS] (all int32 but the
        pool; control[1] is the number of free pages)."""
        self = cls.__new__(cls)
        self._set(pool, block_table, page_count, ref_count, free_list, control)
        return self

    def _set(self, pool, block_table, page_count, ref_count, free_list, control):
        torch = _torch()
        if pool.dim() != 6 or pool.shape[1] != 2:
            raise ValueError("pool must be [layers, 2, num_pages, kv_heads, page_size, head_dim]")
        if pool.dtype not in (torch.float32, torch.bfloat16):
            raise TypeError(f"expected float32 or bfloat16, got {pool.dtype}")
        if block_table.dim() != 2:
            raise ValueError("block_table must be [max_seqs, max_pages]")
        layers, _, num_pages, kv_heads, page_size, head_dim = pool.shape
        max_seqs, max_pages = block_table.shape
        for name, t, shape in (("block_table", block_table, (max_seqs, max_pages)),
                               ("page_count", page_count, (max_seqs,)),
                               ("ref_count", ref_count, (num_pages,)),
                               ("free_list", free_list, (num_pages,)),
                               ("control", control, (CONTROL_WORDS,))):
            if t.dtype != torch.int32 or tuple(t.shape) != shape:
                raise TypeError(f"{name} must be int32 {list(shape)}")
            if t.device != pool.device:
                raise ValueError("all tensors of a cache must be on one device")
        for t in (pool, block_table, page_count, ref_count, free_list, control):
            if not t.is_contiguous():
                raise ValueError("all tensors must be contiguous")
        self.pool, self.block_table, self.page_count = pool, block_table, page_count
        self.ref_count, self.free_list, self.control = ref_count, free_list, control
        self.layers, self.num_pages, self.kv_heads = layers, num_pages, kv_heads
        self.page_size, self.head_dim = page_size, head_dim
        self.max_seqs, self.max_pages = max_seqs, max_pages
        self.device, self.dtype = pool.device, pool.dtype
        self.buffer = control  # the device error word (read_device_error)
        self._struct = _lib.CacheStruct(
            pool.data_ptr(), F32 if pool.dtype == torch.float32 else BF16, layers,
            num_pages, kv_heads, page_size, head_dim, max_seqs, max_pages,
            block_table.data_ptr(), page_count.data_ptr(), ref_count.data_ptr(),
            free_list.data_ptr(), control.data_ptr())
        self._ref = ctypes.byref(self._struct)

    def _current(self):
        """Makes the cache's device the current one for a launch."""
        torch = _torch()
        if self.device.type != "cuda":
            raise ValueError("the cache is not on a CUDA device")
        if self.device.index in (None, torch.cuda.current_device()):
            return _NOTHING
        return torch.cuda.device(self.device)

    def _stream(self, stream) -> int:
        if stream is None:
            stream = _torch().cuda.current_stream(self.device)
        return stream.cuda_stream


class _Nothing:
    def __enter__(self):
        return self

    def __exit__(self, *exc):
        return False


_NOTHING = _Nothing()


def _check(fn: str, status: int) -> None:
    if status != 0:
        raise DsparkError(fn, status)


def _ints(cache, **tensors):
    """int32 vectors [B], contiguous, on the cache's device (None passes)."""
    torch = _torch()
    B = None
    for name, t in tensors.items():
        if t is None:
            continue
        if B is None:
            B = t.shape[0] if t.dim() else 0
        if t.dtype != torch.int32 or t.dim() != 1 or t.shape[0] != B:
            raise TypeError(f"{name} must be int32 [B]")
        if not t.is_contiguous():
            raise ValueError("all tensors must be contiguous")
        if t.device != cache.device:
            raise ValueError(f"{name} must be on the cache's device")
    return B


def _same(cache, name, t, shape, dtype):
    if t.dtype != dtype or t.shape != shape:
        raise TypeError(f"{name} must be {dtype} {list(shape)}")
    if not t.is_contiguous():
        raise ValueError("all tensors must be contiguous")
    if t.device != cache.device:
        raise ValueError(f"{name} must be on the cache's device")


def cache_reserve(cache: PagedCache, length, tokens: int, *, seq=None, stream=None) -> None:
    """Pages for ``tokens`` more tokens of each sequence: length [B] int32
    committed tokens, seq [B] int32 or None (sequences 0..B-1)."""
    B = _ints(cache, length=length, seq=seq)
    with cache._current():
        _check("dspark_cache_reserve", _lib.load().dspark_cache_reserve(
            cache._ref, _ptr(seq), length.data_ptr(), tokens, B, cache._stream(stream)))


def cache_release(cache: PagedCache, seq, *, stream=None) -> None:
    """The sequences seq [B] int32 give up all their pages."""
    B = _ints(cache, seq=seq)
    with cache._current():
        _check("dspark_cache_release", _lib.load().dspark_cache_release(
            cache._ref, seq.data_ptr(), B, cache._stream(stream)))


def cache_fork(cache: PagedCache, parent, child, length, *, stream=None) -> None:
    """Sequence child[b] becomes a copy of the first length[b] tokens of
    parent[b]: full pages are shared, a partly filled one is copied."""
    B = _ints(cache, parent=parent, child=child, length=length)
    with cache._current():
        _check("dspark_cache_fork", _lib.load().dspark_cache_fork(
            cache._ref, parent.data_ptr(), child.data_ptr(), length.data_ptr(), B,
            cache._stream(stream)))


def cache_accept(cache: PagedCache, length, accepted_len, tokens: int, *, path=None,
                 extra: int = 1, seq=None, new_length=None, stream=None):
    """Keeps accepted_len[b] + extra of the ``tokens`` tokens behind the
    committed ones (path [B, P] int32: which ones; None: the first) and gives
    up the pages behind them.  Returns new_length [B] int32."""
    torch = _torch()
    B = _ints(cache, length=length, accepted_len=accepted_len, seq=seq, new_length=new_length)
    width = 0
    if path is not None:
        if path.dim() != 2:
            raise TypeError("path must be int32 [B, P]")
        width = path.shape[1]
        _same(cache, "path", path, (B, width), torch.int32)
    if new_length is None:
        new_length = torch.empty_like(length)
    with cache._current():
        _check("dspark_cache_accept", _lib.load().dspark_cache_accept(
            cache._ref, _ptr(seq), length.data_ptr(), accepted_len.data_ptr(), _ptr(path),
            width, extra, tokens, B, new_length.data_ptr(), cache._stream(stream)))
    return new_length


def _token_stride(name, t, B, T, D) -> int:
    """Elements between consecutive tokens of a [B, T, heads, D] view whose
    heads are dense and whose tokens are evenly spaced."""
    st = t.stride()
    if st[3] != 1 or (t.shape[2] > 1 and st[2] != D):
        raise ValueError(f"{name}: a token's heads must be dense")
    step = st[1] if T > 1 else st[0] if B > 1 else t.shape[2] * D
    if B > 1 and T > 1 and st[0] != T * step:
        raise ValueError(f"{name}: tokens must be evenly spaced")
    return step


def cache_append(cache: PagedCache, layer: int, q, k, v, length, *, position, cos_sin,
                 q_weight=None, k_weight=None, eps: float = 1e-6, interleaved: bool = False,
                 token_count=None, seq=None, q_out=None, stream=None):
    """Normalises and rotates the queries q [B, T, heads, D] and keys k
    [B, T, kv_heads, D] of new tokens and stores the keys and values v at
    places length[b] + t of ``layer`` (their pages must be reserved).  q, k
    and v may be parts of one projection's output.  position [B, T] int32
    rows of cos_sin [max_position, rot_dim] float32 (cosines, then sines);
    q_weight and k_weight [D] float32 or None.  Returns q_out."""
    torch = _torch()
    if q.dim() != 4:
        raise ValueError("q must be [B, T, heads, D]")
    B, T, heads, D = q.shape
    kv = (B, T, cache.kv_heads, cache.head_dim)
    if D != cache.head_dim or k.shape != kv or v.shape != kv:
        raise ValueError("q must be [B, T, heads, D], k and v [B, T, kv_heads, D]")
    dtype, device = cache.dtype, cache.device
    if q.dtype != dtype or k.dtype != dtype or v.dtype != dtype:
        raise TypeError("q, k and v must have the cache's dtype")
    if q.device != device or k.device != device or v.device != device:
        raise ValueError("q, k and v must be on the cache's device")
    if _ints(cache, length=length, token_count=token_count, seq=seq) != B:
        raise TypeError("length must be int32 [B]")
    _same(cache, "position", position, (B, T), torch.int32)
    if cos_sin.dim() != 2:
        raise TypeError("cos_sin must be float32 [max_position, rot_dim]")
    _same(cache, "cos_sin", cos_sin, cos_sin.shape, torch.float32)
    for name, w in (("q_weight", q_weight), ("k_weight", k_weight)):
        if w is not None:
            _same(cache, name, w, (D,), torch.float32)
    if q_out is None:
        q_out = torch.empty((B, T, heads, D), dtype=dtype, device=device)
    else:
        _same(cache, "q_out", q_out, (B, T, heads, D), dtype)
    with cache._current():
        _check("dspark_cache_append", _lib.load().dspark_cache_append(
            cache._ref, layer, _ptr(seq), length.data_ptr(), _ptr(token_count),
            q.data_ptr(), _token_stride("q", q, B, T, D),
            k.data_ptr(), _token_stride("k", k, B, T, D),
            v.data_ptr(), _token_stride("v", v, B, T, D),
            _ptr(q_weight), _ptr(k_weight), eps, cos_sin.data_ptr(), cos_sin.shape[0],
            cos_sin.shape[1], int(interleaved), position.data_ptr(), B, T, heads,
            q_out.data_ptr(), cache._stream(stream)))
    return q_out


class TreeWorkspace:
    """Device scratch for tree_attention, sized for (B, T, heads, kv_heads,
    head_dim) or anything smaller in B and T."""

    def __init__(self, B: int, T: int, heads: int, kv_heads: int, head_dim: int, device=None):
        n = int(_lib.load().dspark_tree_workspace_bytes(B, T, heads, kv_heads, head_dim))
        if n == 0:
            raise DsparkError("dspark_tree_workspace_bytes", 2)
        self.nbytes = n
        self.buffer = _torch().empty(n, dtype=_torch().uint8, device=device or "cuda")


def tree_attention(cache: PagedCache, layer: int, q, length, *, mask=None, token_count=None,
                   position=None, window: int = 0, scale: Optional[float] = None, seq=None,
                   out=None, lse=None, with_lse: bool = False,
                   workspace: Optional[TreeWorkspace] = None, stream=None):
    """Attention of drafted tokens q [B, T, heads, D] over the cache of
    ``layer``, their own keys and values (cache_append) included: all
    committed tokens (the last ``window`` positions if given), and the drafted
    tokens that mask allows: int64 words [B, T] or [T], bit j of word t says
    that token t sees drafted token j (None: tokens 0..t).  scale defaults to
    1 / sqrt(D).  Returns (out, lse); lse is None unless asked for."""
    torch = _torch()
    if q.dim() != 4:
        raise ValueError("q must be [B, T, heads, D]")
    B, T, heads, D = q.shape
    _same(cache, "q", q, (B, T, heads, cache.head_dim), cache.dtype)
    if _ints(cache, length=length, token_count=token_count, seq=seq) != B:
        raise TypeError("length must be int32 [B]")
    stride = 0
    if mask is not None:
        _same(cache, "mask", mask, (T,) if mask.dim() == 1 else (B, T), torch.int64)
        stride = T if mask.dim() == 2 else 0
    if position is not None:
        _same(cache, "position", position, (B, T), torch.int32)
    if out is None:
        out = torch.empty_like(q)
    else:
        _same(cache, "out", out, (B, T, heads, D), cache.dtype)
    if lse is not None:
        _same(cache, "lse", lse, (B, T, heads), torch.float32)
    elif with_lse:
        lse = torch.empty((B, T, heads), dtype=torch.float32, device=cache.device)
    if workspace is None:
        workspace = TreeWorkspace(B, T, heads, cache.kv_heads, D, device=cache.device)
    elif workspace.buffer.device != cache.device:
        raise ValueError("workspace must be on the cache's device")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    with cache._current():
        _check("dspark_tree_attention", _lib.load().dspark_tree_attention(
            cache._ref, layer, _ptr(seq), length.data_ptr(), _ptr(token_count),
            q.data_ptr(), _ptr(mask), stride, _ptr(position), window, scale, B, T, heads,
            out.data_ptr(), _ptr(lse), workspace.buffer.data_ptr(), workspace.nbytes,
            cache._stream(stream)))
    return out, lse
