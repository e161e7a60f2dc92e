"""CPU-only checks of the calls that read part of the cache: what they refuse,
with a status and before any launch (the fake device addresses are never read),
and what the Python functions refuse."""
import ctypes

import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.test_cache_abi import (BAD_CACHES, FAKE, INVALID, UNSUPPORTED, WORKSPACE, host_cache, lib, struct)  # noqa: F401


def bounds(lib, c=None, **over):
    a = dict(c=c or ctypes.byref(struct()), seq=None, start=FAKE, length=FAKE, B=2, bounds=FAKE)
    a.update(over)
    return lib.dspark_cache_bounds(a["c"], a["seq"], a["start"], a["length"], a["B"], a["bounds"], None)


def select(lib, c=None, **over):
    c = c or ctypes.byref(struct())
    a = dict(layer=0, seq=None, length=FAKE, tokens=None, q=FAKE, bounds=FAKE, count=4, first=0, last=0, shared=0,
             B=2, T=4, heads=4, pages=FAKE, ws=FAKE,
             bytes=lib.dspark_select_workspace_bytes(ctypes.byref(struct()), 2, 4, 0))
    a.update(over)
    return lib.dspark_select_pages(
        c, a["layer"], a["seq"], a["length"], a["tokens"], a["q"], a["bounds"], a["count"], a["first"], a["last"],
        a["shared"], a["B"], a["T"], a["heads"], a["pages"], a["ws"], a["bytes"], None)


def attention(lib, fn, c=None, **over):
    """dspark_sparse_attention or dspark_prefix_attention."""
    c = c or ctypes.byref(struct())
    B, T, heads = over.get("B", 2), over.get("T", 4), over.get("heads", 4)
    b, t = max(1, min(B, 1024)), max(1, min(T, 64))
    if fn == "sparse":
        nbytes = lib.dspark_sparse_workspace_bytes(ctypes.byref(struct()), b, t, 4, 5)
    else:
        nbytes = lib.dspark_prefix_workspace_bytes(b, t, 4, 2, 64)
    a = dict(layer=0, seq=None, length=FAKE, count=None, q=FAKE, pages=FAKE, width=5, shared=0, start=FAKE, prefix=FAKE,
             groups=1, mask=None, stride=0, scale=0.1, out=FAKE + (1 << 30), lse=None, ws=FAKE, bytes=nbytes)
    a.update(over)
    special = ((a["pages"], a["width"], a["shared"]) if fn == "sparse" else (a["start"], a["prefix"], a["groups"]))
    return getattr(lib, f"dspark_{fn}_attention")(
        c, a["layer"], a["seq"], a["length"], a["count"], a["q"], *special, a["mask"], a["stride"], a["scale"],
        B, T, heads, a["out"], a["lse"], a["ws"], a["bytes"], None)


BOTH = ("sparse", "prefix")


@pytest.mark.parametrize("over,want", BAD_CACHES)
def test_every_call_checks_the_cache(lib, over, want):
    c = ctypes.byref(struct(**over))
    assert bounds(lib, c=c) == want and select(lib, c=c) == want
    assert all(attention(lib, fn, c=c) == want for fn in BOTH)
    assert lib.dspark_select_workspace_bytes(c, 2, 4, 0) == 0
    assert lib.dspark_sparse_workspace_bytes(c, 2, 4, 4, 5) == 0


@pytest.mark.parametrize("B,want", [(0, INVALID), (-3, INVALID), (1025, UNSUPPORTED)])
def test_batch_limits(lib, B, want):
    assert bounds(lib, B=B) == want and select(lib, B=B) == want
    assert all(attention(lib, fn, B=B) == want for fn in BOTH)
    assert lib.dspark_select_workspace_bytes(ctypes.byref(struct()), B, 4, 0) == 0


@pytest.mark.parametrize("over", [dict(start=None), dict(length=None), dict(bounds=None), dict(seq=FAKE + 2),
                                  dict(start=FAKE + 1), dict(length=FAKE + 2), dict(bounds=FAKE + 8)])
def test_bounds_refuses(lib, over):
    assert bounds(lib, **over) == INVALID


@pytest.mark.parametrize("over,want", [
    (dict(length=None), INVALID), (dict(q=None), INVALID), (dict(bounds=None), INVALID), (dict(pages=None), INVALID),
    (dict(layer=2), INVALID), (dict(layer=-1), INVALID), (dict(T=0), INVALID), (dict(heads=5), INVALID),
    (dict(heads=0), INVALID), (dict(count=0), INVALID), (dict(first=-1), INVALID), (dict(last=-1), INVALID),
    (dict(first=5), INVALID), (dict(first=2, last=3), INVALID), (dict(first=2 ** 31 - 1, last=2 ** 31 - 1), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(bounds=FAKE + 8), INVALID), (dict(pages=FAKE + 2), INVALID),
    (dict(tokens=FAKE + 1), INVALID), (dict(seq=FAKE + 1), INVALID), (dict(T=65), UNSUPPORTED),
    (dict(heads=66), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 64), WORKSPACE),
    (dict(bytes=1000), WORKSPACE), (dict(shared=1, bytes=100), WORKSPACE),
])
def test_select_refuses(lib, over, want):
    assert select(lib, **over) == want


def test_select_workspace_bytes(lib):
    c = ctypes.byref(struct())
    f = lib.dspark_select_workspace_bytes
    assert 0 < f(c, 2, 4, 1) < f(c, 2, 4, 0) and f(c, 2, 4, 0) % 256 == 0
    assert f(c, 2, 65, 0) == 0 and f(c, 2, 0, 0) == 0
    assert f(ctypes.byref(struct(kv_heads=1024, max_seqs=1, max_pages=1 << 27, page_size=1)), 1024, 1, 0) == 0


@pytest.mark.parametrize("fn", BOTH)
@pytest.mark.parametrize("over,want", [
    (dict(length=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID), (dict(layer=2), INVALID),
    (dict(layer=-1), INVALID), (dict(scale=float("inf")), INVALID), (dict(scale=float("nan")), INVALID),
    (dict(T=0), INVALID), (dict(heads=5), INVALID), (dict(heads=0), INVALID), (dict(mask=FAKE + 4), INVALID),
    (dict(mask=FAKE, stride=3), INVALID), (dict(mask=FAKE, stride=-1), INVALID), (dict(q=FAKE + 8), INVALID),
    (dict(out=FAKE + 8), INVALID), (dict(out=FAKE), INVALID), (dict(out=FAKE + 16), INVALID), (dict(lse=FAKE + 1), INVALID),
    (dict(seq=FAKE + 2), INVALID), (dict(count=FAKE + 2), INVALID), (dict(T=65), UNSUPPORTED),
    (dict(heads=66), UNSUPPORTED), (dict(ws=None), WORKSPACE), (dict(ws=FAKE + 64), WORKSPACE),
    (dict(bytes=1000), WORKSPACE),
])
def test_attentions_refuse(lib, fn, over, want):
    assert attention(lib, fn, **over) == want


@pytest.mark.parametrize("over,want", [
    (dict(pages=None), INVALID), (dict(pages=FAKE + 2), INVALID), (dict(width=0), INVALID), (dict(width=-1), INVALID),
    (dict(width=1 << 23), UNSUPPORTED)])
def test_sparse_refuses(lib, over, want):
    assert attention(lib, "sparse", **over) == want


@pytest.mark.parametrize("over,want", [
    (dict(start=None), INVALID), (dict(prefix=None), INVALID), (dict(start=FAKE + 2), INVALID),
    (dict(prefix=FAKE + 1), INVALID), (dict(groups=0), INVALID), (dict(groups=-1), INVALID), (dict(groups=3), INVALID)])
def test_prefix_refuses(lib, over, want):
    assert attention(lib, "prefix", **over) == want


def test_attention_workspace_bytes(lib):
    c = ctypes.byref(struct(max_pages=4096, page_size=16))
    f = lib.dspark_sparse_workspace_bytes
    assert f(c, 2, 4, 4, 100) > f(c, 2, 4, 4, 10) > 0 and f(c, 2, 4, 4, 100) >= f(c, 1, 4, 4, 100)
    assert f(c, 2, 4, 4, 5000) == f(c, 2, 4, 4, 6000)  # a list names no page twice
    for bad in [(0, 4, 4, 5), (2, 0, 4, 5), (2, 65, 4, 5), (2, 4, 5, 5), (2, 4, 66, 5), (2, 4, 4, 0), (1025, 4, 4, 5)]:
        assert f(c, *bad) == 0, bad
    f = lib.dspark_prefix_workspace_bytes
    assert f(88, 8, 32, 8, 128) > f(8, 4, 32, 8, 128) > 0 and f(88, 8, 32, 8, 128) % 256 == 0
    for bad in [(0, 8, 32, 8, 128), (8, 0, 32, 8, 128), (8, 65, 32, 8, 128), (8, 8, 33, 8, 128), (8, 8, 66, 2, 128),
                (8, 8, 32, 8, 260), (8, 8, 32, 8, 100), (2000, 8, 32, 8, 128), (8, 8, 32, 0, 128)]:
        assert f(*bad) == 0, bad


def test_python_refuses_tensors_that_do_not_fit(lib):
    c = host_cache()
    i32 = torch.int32
    one, q = torch.zeros(1, dtype=i32), torch.zeros(1, 3, 4, 8)
    b = torch.zeros(1, 6, 2, 2, 8)
    with pytest.raises(ValueError):  # a cache in host memory is not launched on
        dspark.cache_bounds(c, one, one, bounds=b)
    for bad in (dict(start=one.long()), dict(length=torch.zeros(2, dtype=i32)), dict(bounds=b[:, :5]),
                dict(bounds=b.double()), dict(bounds=b.transpose(3, 4).contiguous().transpose(3, 4)), dict(seq=one.long())):
        a = dict(start=one, length=one, bounds=b) | bad
        with pytest.raises((TypeError, ValueError)):
            dspark.cache_bounds(c, a.pop("start"), a.pop("length"), **a)
    for bad in (dict(q=q[0]), dict(q=q.double()), dict(bounds=b[0]), dict(length=one.long()),
                dict(pages=torch.zeros(1, 3, 2, 5, dtype=i32)), dict(pages=torch.zeros(1, 3, 2, 4)),
                dict(pages=torch.zeros(1, 3, 2, 4, dtype=i32), shared=True), dict(token_count=one.long())):
        a = dict(bounds=b, q=q, length=one, pages=torch.zeros(1, 3, 2, 4, dtype=i32)) | bad
        with pytest.raises((TypeError, ValueError)):
            dspark.select_pages(c, 0, a.pop("bounds"), a.pop("q"), a.pop("length"), 4, **a)
    pages, start = torch.zeros(1, 3, 2, 5, dtype=i32), torch.zeros(2, dtype=i32)
    for bad in (dict(q=q.double()), dict(q=q[0]), dict(mask=torch.zeros(3)), dict(lse=torch.zeros(1, 3)),
                dict(mask=torch.zeros(2, 3, dtype=torch.int64)), dict(out=q[:, :2]), dict(length=one.long()),
                dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), dict(token_count=start)):
        for fn, more in ((dspark.sparse_attention, (pages,)), (dspark.prefix_attention, (start, one))):
            a = dict(q=q, length=one) | bad
            with pytest.raises((TypeError, ValueError)):
                fn(c, 0, a.pop("q"), a.pop("length"), *more, **a)
    for bad in (pages[0], pages.long(), pages[:, :2], pages[:, :, :1], pages.transpose(1, 2)):
        with pytest.raises((TypeError, ValueError)):
            dspark.sparse_attention(c, 0, q, one, bad)
    for bad in ((start.long(), one), (start[:1], one), (start, one.long()), (start, start), (start[None], one)):
        with pytest.raises((TypeError, ValueError)):
            dspark.prefix_attention(c, 0, q, one, *bad)


def test_prefix_workspace_bytes_goes_by_the_calls_limits(lib):
    """B * T * heads < 2^31, in the size as in the call."""
    f = lib.dspark_prefix_workspace_bytes
    assert f(1024, 64, 32768, 1024, 8) == 0
    assert f(1023, 64, 32768, 1024, 8) > 0
    c = ctypes.byref(struct(kv_heads=1024, head_dim=8, max_seqs=1))
    assert attention(lib, "prefix", c=c, B=1024, T=64, heads=32768, bytes=1 << 62, out=FAKE + (1 << 50)) == UNSUPPORTED
