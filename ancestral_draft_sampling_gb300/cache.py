"""The paged key/value cache and the attention of drafted tokens over it, for
torch tensors: checks of dtypes, shapes and devices, and raw pointers to the
library.  The layouts, limits and device errors are described in
include/dspark.h."""
from __future__ import annotations

import contextlib
import ctypes
import math
from typing import Optional

import torch

from . import _lib
from ._lib import BF16, F32, DsparkError

CONTROL_WORDS = 64 + 2 * 1024  # DSPARK_CACHE_CONTROL_WORDS


# The current device and a device's current stream, as a number: torch's own
# functions behind the public ones, which cost less, where it has them.
_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device
_stream_of = (getattr(torch._C, "_cuda_getCurrentRawStream", None)
              or (lambda index: torch.cuda.current_stream(index).cuda_stream))
_here = contextlib.nullcontext()


def _on(stream):
    """Memory that a call makes belongs to the stream that the call runs on:
    the allocator hands it out again only behind the call's kernels."""
    return _here if stream is None else torch.cuda.stream(stream)


class PagedCache:
    """A paged key/value cache: ``pool`` [layers, 2, num_pages, kv_heads,
    page_size, head_dim], float32 or bfloat16, and the tables that say which
    sequence holds which page.  A new cache is empty: cache_reserve gives its
    sequences pages.  The lengths of the sequences are the caller's."""

    def __init__(self, layers: int, num_pages: int, page_size: int, kv_heads: int,
                 head_dim: int, max_seqs: int, max_pages: int, dtype=None,
                 device=None, stream=None):
        device = device or "cuda"
        i32 = dict(dtype=torch.int32, device=device)
        with _on(stream):
            self._set(torch.empty(layers, 2, num_pages, kv_heads, page_size, head_dim,
                                  dtype=dtype or torch.bfloat16, device=device),
                      torch.empty(max_seqs, max_pages, **i32), torch.empty(max_seqs, **i32),
                      torch.empty(num_pages, **i32), torch.empty(num_pages, **i32),
                      torch.empty(CONTROL_WORDS, **i32))
        _call(self, "dspark_cache_init", stream)

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
        self.index = pool.get_device()  # -1 on the host
        self.buffer = control  # the device error word (read_device_error)
        self._struct = _lib.CacheStruct(
            pool.data_ptr(), F32 if pool.dtype == torch.float32 else BF16, layers,
            num_pages, kv_heads, page_size, head_dim, max_seqs, max_pages,
            block_table.data_ptr(), page_count.data_ptr(), ref_count.data_ptr(),
            free_list.data_ptr(), control.data_ptr())
        self._ref = ctypes.byref(self._struct)


_functions = {}  # of the library, by name


def _call(cache, fn, stream, *args):
    """Calls the library on the cache's device and on `stream` (None: that
    device's current stream)."""
    call = _functions.get(fn)
    if call is None:
        call = _functions[fn] = getattr(_lib.load(), fn)
    index = cache.index
    if index < 0:
        raise ValueError("the cache is not on a CUDA device")
    if index == _device():
        status = call(cache._ref, *args,
                      _stream_of(index) if stream is None else stream.cuda_stream)
    else:
        with torch.cuda.device(index):
            status = call(cache._ref, *args,
                          _stream_of(index) if stream is None else stream.cuda_stream)
    if status != 0:
        raise DsparkError(fn, status)


def _bad(cache, name, t, dtype, shape):
    """Says what is wrong with a tensor that _ptr_of refused."""
    if t.dtype != dtype or t.shape != tuple(shape):
        raise TypeError(f"{name} must be {str(dtype)[6:]} {list(shape)}")
    if not t.is_contiguous():
        raise ValueError(f"all tensors must be contiguous: {name} is not")
    raise ValueError(f"{name} must be on the cache's device")


def _ptr_of(cache, name, t, dtype, shape) -> Optional[int]:
    """The address of a tensor of this dtype and shape, contiguous on the
    cache's device; None stays None."""
    if t is None:
        return None
    if (t.dtype is not dtype or t.shape != shape or not t.is_contiguous()
            or t.get_device() != cache.index):
        _bad(cache, name, t, dtype, shape)
    return t.data_ptr()


def _batch(length) -> int:
    if length.dim() != 1:
        raise TypeError("the sequences of a call are int32 [B]")
    return length.shape[0]


def cache_reserve(cache: PagedCache, length, tokens: int, *, seq=None, stream=None) -> None:
    """Pages for ``tokens`` more tokens of each sequence: length [B] int32
    committed tokens, seq [B] int32 or None (sequences 0..B-1)."""
    i32, shape = torch.int32, (_batch(length),)
    _call(cache, "dspark_cache_reserve", stream, _ptr_of(cache, "seq", seq, i32, shape),
          _ptr_of(cache, "length", length, i32, shape), tokens, shape[0])


def cache_release(cache: PagedCache, seq, *, stream=None) -> None:
    """The sequences seq [B] int32 give up all their pages."""
    i32, shape = torch.int32, (_batch(seq),)
    _call(cache, "dspark_cache_release", stream, _ptr_of(cache, "seq", seq, i32, shape), shape[0])


def cache_fork(cache: PagedCache, parent, child, length, *, stream=None) -> None:
    """Sequence child[b] becomes a copy of the first length[b] tokens of
    parent[b]: full pages are shared, a partly filled one is copied."""
    i32, shape = torch.int32, (_batch(length),)
    _call(cache, "dspark_cache_fork", stream, _ptr_of(cache, "parent", parent, i32, shape),
          _ptr_of(cache, "child", child, i32, shape),
          _ptr_of(cache, "length", length, i32, shape), shape[0])


def cache_accept(cache: PagedCache, length, accepted_len, tokens: int, *, path=None,
                 extra: int = 1, seq=None, new_length=None, stream=None):
    """Keeps accepted_len[b] + extra of the ``tokens`` tokens behind the
    committed ones (path [B, P] int32: which ones; None: the first) and gives
    up the pages behind them.  Returns new_length [B] int32."""
    i32, shape = torch.int32, (_batch(length),)
    width = 0
    if path is not None:
        if path.dim() != 2:
            raise TypeError("path must be int32 [B, P]")
        width = path.shape[1]
    at = _ptr_of(cache, "length", length, i32, shape)
    if new_length is None:
        with _on(stream):
            new_length = torch.empty(shape, dtype=i32, device=cache.device)
    _call(cache, "dspark_cache_accept", stream, _ptr_of(cache, "seq", seq, i32, shape), at,
          _ptr_of(cache, "accepted_len", accepted_len, i32, shape),
          _ptr_of(cache, "path", path, i32, (shape[0], width)), width, extra, tokens, shape[0],
          _ptr_of(cache, "new_length", new_length, i32, shape))
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
    if q.dim() != 4:
        raise ValueError("q must be [B, T, heads, D]")
    B, T, heads, D = q.shape
    kv = (B, T, cache.kv_heads, cache.head_dim)
    if D != cache.head_dim or k.shape != kv or v.shape != kv:
        raise ValueError("q must be [B, T, heads, D], k and v [B, T, kv_heads, D]")
    dtype, index = cache.dtype, cache.index
    if not (q.dtype is dtype and k.dtype is dtype and v.dtype is dtype):
        raise TypeError("q, k and v must have the cache's dtype")
    if not (q.get_device() == index and k.get_device() == index and v.get_device() == index):
        raise ValueError("q, k and v must be on the cache's device")
    if cos_sin.dim() != 2:
        raise TypeError("cos_sin must be float32 [max_position, rot_dim]")
    if q_out is None:
        with _on(stream):
            q_out = torch.empty((B, T, heads, D), dtype=dtype, device=cache.device)
    i32, f32, shape = torch.int32, torch.float32, (B,)
    _call(cache, "dspark_cache_append", stream, layer, _ptr_of(cache, "seq", seq, i32, shape),
          _ptr_of(cache, "length", length, i32, shape),
          _ptr_of(cache, "token_count", token_count, i32, shape),
          q.data_ptr(), _token_stride("q", q, B, T, D),
          k.data_ptr(), _token_stride("k", k, B, T, D),
          v.data_ptr(), _token_stride("v", v, B, T, D),
          _ptr_of(cache, "q_weight", q_weight, f32, (D,)),
          _ptr_of(cache, "k_weight", k_weight, f32, (D,)), eps,
          _ptr_of(cache, "cos_sin", cos_sin, f32, cos_sin.shape), cos_sin.shape[0],
          cos_sin.shape[1], 1 if interleaved else 0,
          _ptr_of(cache, "position", position, i32, (B, T)), B, T, heads,
          _ptr_of(cache, "q_out", q_out, dtype, (B, T, heads, D)))
    return q_out


class TreeWorkspace:
    """Device scratch for tree_attention, sized for (B, T, heads, kv_heads,
    head_dim) or anything smaller in B and T."""

    def __init__(self, B: int, T: int, heads: int, kv_heads: int, head_dim: int, device=None):
        n = int(_lib.load().dspark_tree_workspace_bytes(B, T, heads, kv_heads, head_dim))
        if n == 0:
            raise DsparkError("dspark_tree_workspace_bytes", 2)
        self.nbytes = n
        self.buffer = torch.empty(n, dtype=torch.uint8, device=device or "cuda")


def tree_attention(cache: PagedCache, layer: int, q, length, *, mask=None, token_count=None,
                   position=None, window: int = 0, scale: Optional[float] = None, seq=None,
                   out=None, lse=None, with_lse: bool = False,
                   workspace: Optional[TreeWorkspace] = None, stream=None):
    """Attention of drafted tokens q [B, T, heads, D] over the cache of
    ``layer``, their own keys and values (cache_append) included: all
    committed tokens (the last ``window`` positions if given), and the drafted
    tokens that mask allows: int64 words [B, T] or [T], bit j of word t says
    that token t sees drafted token j (None: tokens 0..t, whatever the window).
    scale defaults to 1 / sqrt(D).  Returns (out, lse); lse is None unless asked for."""
    if q.dim() != 4:
        raise ValueError("q must be [B, T, heads, D]")
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
    if workspace is None:
        with _on(stream):
            workspace = TreeWorkspace(B, T, heads, cache.kv_heads, D, device=cache.device)
    elif workspace.buffer.get_device() != cache.index:
        raise ValueError("workspace must be on the cache's device")
    if scale is None:
        scale = 1.0 / math.sqrt(D)
    i32, shape = torch.int32, (B,)
    _call(cache, "dspark_tree_attention", stream, layer, _ptr_of(cache, "seq", seq, i32, shape),
          _ptr_of(cache, "length", length, i32, shape),
          _ptr_of(cache, "token_count", token_count, i32, shape), at,
          _ptr_of(cache, "mask", mask, torch.int64, (B, T) if stride else (T,)), stride,
          _ptr_of(cache, "position", position, i32, (B, T)), window, scale, B, T, heads,
          _ptr_of(cache, "out", out, cache.dtype, full),
          _ptr_of(cache, "lse", lse, torch.float32, (B, T, heads)),
          workspace.buffer.data_ptr(), workspace.nbytes)
    return out, lse
