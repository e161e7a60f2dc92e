"""CPU-only checks of the paged cache's entry points: what they refuse, with a
status and before any launch (the fake device addresses are never read), and
what the Python functions refuse."""
import ctypes

import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from ancestral_draft_sampling_gb300 import _lib

FAKE = 0x7F0000000000
OK, INVALID, UNSUPPORTED, WORKSPACE = 0, 1, 2, 3


@pytest.fixture(scope="module")
def lib():
    import __graft_entry__
    __graft_entry__.build_library()
    return _lib.load()


def struct(**over):
    a = dict(pool=FAKE, dtype=1, layers=2, num_pages=10, kv_heads=2, page_size=16,
             head_dim=64, max_seqs=4, max_pages=8, block_table=FAKE, page_count=FAKE,
             ref_count=FAKE, free_list=FAKE, control=FAKE)
    a.update(over)
    return _lib.CacheStruct(*[a[n] for n, _ in _lib.CacheStruct._fields_])


BAD_CACHES = [
    (dict(pool=None), INVALID), (dict(block_table=None), INVALID),
    (dict(page_count=None), INVALID), (dict(ref_count=None), INVALID),
    (dict(free_list=None), INVALID), (dict(control=None), INVALID),
    (dict(dtype=2), INVALID), (dict(layers=0), INVALID), (dict(num_pages=0), INVALID),
    (dict(kv_heads=-1), INVALID), (dict(page_size=0), INVALID), (dict(head_dim=0), INVALID),
    (dict(max_seqs=0), INVALID), (dict(max_pages=0), INVALID), (dict(pool=FAKE + 8), INVALID),
    (dict(control=FAKE + 4), INVALID), (dict(block_table=FAKE + 2), INVALID),
    (dict(head_dim=12), UNSUPPORTED), (dict(head_dim=264), UNSUPPORTED),
    (dict(layers=1025), UNSUPPORTED), (dict(page_size=4097), UNSUPPORTED),
    (dict(max_seqs=1 << 20, max_pages=1 << 11), UNSUPPORTED),
    (dict(max_seqs=1, max_pages=1 << 20, page_size=2048), UNSUPPORTED),
]


@pytest.mark.parametrize("over,want", BAD_CACHES)
def test_every_call_checks_the_cache(lib, over, want):
    c = ctypes.byref(struct(**over))
    assert lib.dspark_cache_init(c, None) == want
    assert lib.dspark_cache_reserve(c, None, FAKE, 1, 1, None) == want
    assert lib.dspark_cache_release(c, None, 1, None) == want
    assert lib.dspark_cache_fork(c, FAKE, FAKE, FAKE, 1, None) == want
    assert lib.dspark_cache_accept(c, None, FAKE, FAKE, None, 0, 1, 4, 1, FAKE, None) == want
    assert append(lib, c=c) == want
    assert attend(lib, c=c) == want


def test_null_cache(lib):
    assert lib.dspark_cache_init(None, None) == INVALID
    assert lib.dspark_cache_release(None, None, 1, None) == INVALID


@pytest.mark.parametrize("B,want", [(0, INVALID), (-3, INVALID), (1025, UNSUPPORTED)])
def test_batch_limits(lib, B, want):
    c = ctypes.byref(struct())
    assert lib.dspark_cache_reserve(c, None, FAKE, 1, B, None) == want
    assert lib.dspark_cache_release(c, None, B, None) == want
    assert lib.dspark_cache_fork(c, FAKE, FAKE, FAKE, B, None) == want
    assert lib.dspark_cache_accept(c, None, FAKE, FAKE, None, 0, 1, 4, B, FAKE, None) == want
    assert append(lib, B=B) == want and attend(lib, B=B) == want


def test_bookkeeping_arguments(lib):
    c = ctypes.byref(struct())
    assert lib.dspark_cache_reserve(c, None, None, 1, 1, None) == INVALID
    assert lib.dspark_cache_reserve(c, None, FAKE, -1, 1, None) == INVALID
    assert lib.dspark_cache_reserve(c, FAKE + 1, FAKE, 1, 1, None) == INVALID
    assert lib.dspark_cache_release(c, FAKE + 2, 1, None) == INVALID
    for i in range(3):
        args = [FAKE, FAKE, FAKE]
        args[i] = None
        assert lib.dspark_cache_fork(c, *args, 1, None) == INVALID
        args[i] = FAKE + 1
        assert lib.dspark_cache_fork(c, *args, 1, None) == INVALID
    good = dict(seq=None, length=FAKE, acc=FAKE, path=FAKE, width=8, extra=1, tokens=8, B=1, new=FAKE)
    for over, want in [(dict(length=None), INVALID), (dict(acc=None), INVALID),
                       (dict(new=None), INVALID), (dict(width=0), INVALID),
                       (dict(extra=-1), INVALID), (dict(tokens=0), INVALID),
                       (dict(path=FAKE + 3), INVALID), (dict(width=65), UNSUPPORTED)]:
        a = {**good, **over}
        assert lib.dspark_cache_accept(c, a["seq"], a["length"], a["acc"], a["path"], a["width"],
                                       a["extra"], a["tokens"], a["B"], a["new"], None) == want


def append(lib, c=None, **over):
    a = dict(c=c or ctypes.byref(struct()), layer=0, seq=None, length=FAKE, count=None, q=FAKE,
             qs=256, k=FAKE, ks=128, v=FAKE, vs=128, wq=None, wk=None, eps=1e-6, cs=FAKE,
             top=10, rot=64, inter=0, pos=FAKE, B=1, T=4, heads=4, out=FAKE + 256)
    a.update(over)
    return lib.dspark_cache_append(
        a["c"], a["layer"], a["seq"], a["length"], a["count"], a["q"], a["qs"], a["k"], a["ks"],
        a["v"], a["vs"], a["wq"], a["wk"], a["eps"], a["cs"], a["top"], a["rot"], a["inter"],
        a["pos"], a["B"], a["T"], a["heads"], a["out"], None)


@pytest.mark.parametrize("over,want", [
    (dict(length=None), INVALID), (dict(q=None), INVALID), (dict(k=None), INVALID),
    (dict(v=None), INVALID), (dict(cs=None), INVALID), (dict(pos=None), INVALID),
    (dict(out=None), INVALID), (dict(layer=2), INVALID), (dict(layer=-1), INVALID),
    (dict(T=0), INVALID), (dict(top=0), INVALID), (dict(rot=0), INVALID), (dict(rot=66), INVALID),
    (dict(rot=7), INVALID), (dict(eps=-1.0), INVALID), (dict(eps=float("nan")), INVALID),
    (dict(q=FAKE + 8), INVALID), (dict(out=FAKE + 2), INVALID), (dict(wq=FAKE + 1), INVALID),
    (dict(heads=3), INVALID), (dict(heads=0), INVALID), (dict(qs=255), INVALID),
    (dict(qs=260), INVALID), (dict(ks=120), INVALID), (dict(vs=0), INVALID),
    (dict(out=FAKE, qs=512), INVALID),   # in place over a wider row
    (dict(B=1024, T=1 << 14), UNSUPPORTED),
])
def test_append_refuses(lib, over, want):
    assert append(lib, **over) == want


def attend(lib, c=None, **over):
    B, T, heads = over.get("B", 2), over.get("T", 4), over.get("heads", 4)
    a = dict(c=c or ctypes.byref(struct()), layer=0, seq=None, length=FAKE, count=None, q=FAKE,
             mask=None, stride=0, pos=None, window=0, scale=0.1, out=FAKE, lse=None, ws=FAKE,
             bytes=lib.dspark_tree_workspace_bytes(max(1, min(B, 1024)), max(1, min(T, 64)), 4, 2, 64))
    a.update(over)
    return lib.dspark_tree_attention(
        a["c"], a["layer"], a["seq"], a["length"], a["count"], a["q"], a["mask"], a["stride"],
        a["pos"], a["window"], a["scale"], B, T, heads, a["out"], a["lse"], a["ws"], a["bytes"], None)


@pytest.mark.parametrize("over,want", [
    (dict(length=None), INVALID), (dict(q=None), INVALID), (dict(out=None), INVALID),
    (dict(layer=2), INVALID), (dict(window=-1), INVALID), (dict(scale=float("inf")), INVALID),
    (dict(T=0), INVALID), (dict(heads=5), INVALID), (dict(mask=FAKE + 4), INVALID),
    (dict(mask=FAKE, stride=3), INVALID), (dict(q=FAKE + 8), INVALID), (dict(lse=FAKE + 1), INVALID),
    (dict(T=65), UNSUPPORTED), (dict(heads=66), UNSUPPORTED), (dict(ws=None), WORKSPACE),
    (dict(ws=FAKE + 64), WORKSPACE), (dict(bytes=1000), WORKSPACE),
])
def test_attention_refuses(lib, over, want):
    assert attend(lib, **over) == want


def test_tree_workspace_bytes(lib):
    f = lib.dspark_tree_workspace_bytes
    assert f(88, 8, 32, 8, 128) > 0 and f(88, 8, 32, 8, 128) % 256 == 0
    assert f(88, 8, 32, 8, 128) >= f(8, 4, 32, 8, 128)
    for bad in [(0, 8, 32, 8, 128), (8, 0, 32, 8, 128), (8, 65, 32, 8, 128), (8, 8, 33, 8, 128),
                (8, 8, 66, 2, 128), (8, 8, 32, 8, 260), (8, 8, 32, 8, 100), (2000, 8, 32, 8, 128)]:
        assert f(*bad) == 0, bad


def host_cache(**over):
    a = dict(pool=torch.zeros(1, 2, 6, 2, 4, 8), block_table=torch.zeros(3, 5, dtype=torch.int32),
             page_count=torch.zeros(3, dtype=torch.int32), ref_count=torch.zeros(6, dtype=torch.int32),
             free_list=torch.zeros(6, dtype=torch.int32),
             control=torch.zeros(64 + 2 * 1024, dtype=torch.int32))
    a.update(over)
    return dspark.PagedCache.from_tensors(**a)


def test_python_refuses_tensors_that_do_not_fit(lib):
    with pytest.raises(ValueError):
        host_cache(pool=torch.zeros(2, 6, 2, 4, 8))
    with pytest.raises(TypeError):
        host_cache(pool=torch.zeros(1, 2, 6, 2, 4, 8, dtype=torch.float16))
    with pytest.raises(TypeError):
        host_cache(ref_count=torch.zeros(5, dtype=torch.int32))
    with pytest.raises(TypeError):
        host_cache(control=torch.zeros(64, dtype=torch.int32))
    with pytest.raises(ValueError):
        host_cache(block_table=torch.zeros(5, 3, dtype=torch.int32).t())
    c = host_cache()
    one = torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):   # a cache in host memory is not launched on
        dspark.cache_reserve(c, one, 1)
    with pytest.raises(TypeError):
        dspark.cache_reserve(c, one.long(), 1)
    with pytest.raises(TypeError):
        dspark.cache_fork(c, one, torch.zeros(2, dtype=torch.int32), one)
    with pytest.raises(TypeError):
        dspark.cache_accept(c, one, one, 3, path=torch.zeros(2, 3, dtype=torch.int32))
    q, kv = torch.zeros(1, 3, 4, 8), torch.zeros(1, 3, 2, 8)
    args = dict(position=torch.zeros(1, 3, dtype=torch.int32), cos_sin=torch.zeros(9, 8))
    for bad in (dict(q=q[0]), dict(k=kv[:, :2]), dict(v=kv.double()), dict(q=q.transpose(1, 2)),
                dict(position=args["position"].long()), dict(cos_sin=args["cos_sin"].double()),
                dict(q_weight=torch.ones(7)), dict(q_out=q[..., :4])):
        a = dict(q=q, k=kv, v=kv, length=one, **args) | bad
        with pytest.raises((TypeError, ValueError)):
            dspark.cache_append(c, 0, a.pop("q"), a.pop("k"), a.pop("v"), a.pop("length"), **a)
    for bad in (dict(q=q.double()), dict(q=q[0]), dict(mask=torch.zeros(3)), dict(lse=torch.zeros(1, 3)),
                dict(mask=torch.zeros(2, 3, dtype=torch.int64)), dict(position=torch.zeros(1, 3)),
                dict(q=q.transpose(2, 3).contiguous().transpose(2, 3)), dict(out=q[:, :2])):
        a = dict(q=q, length=one) | bad
        with pytest.raises((TypeError, ValueError)):
            dspark.tree_attention(c, 0, a.pop("q"), a.pop("length"), **a)
