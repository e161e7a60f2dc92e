"""Reading part of a cache whose pages and bounds lie more than 4 GB from where
they begin, and calls that share a workspace made for larger ones."""
import math

import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.cache_ref import attend_bounds, place, tree_sees
from tests.test_gpu_tree_units import attend_all

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def calls(c, length, start, prefix, q, count, ws={}):
    """All four of them; what they return."""
    n = len(length)
    length = ints(length)
    bounds = dspark.cache_bounds(c, ints([0] * n), length)
    pages = dspark.select_pages(c, 0, bounds, q, length, count, first=1, last=1, workspace=ws.get("select"))
    sparse = dspark.sparse_attention(c, 0, q, length, pages, with_lse=True, workspace=ws.get("sparse"))
    shared = dspark.prefix_attention(c, 0, q, length, ints(start), ints(prefix), with_lse=True,
                                     workspace=ws.get("prefix"))
    assert dspark.read_device_error(c) == 0
    return bounds, pages, *sparse, *shared


def small_cache(dtype, page, D, kv, seed):
    """Three sequences, the second a fork of the first at 500 tokens; 600 pages."""
    g = torch.Generator(device="cuda").manual_seed(seed)
    c = dspark.PagedCache(1, 600, page, kv, D, 4, 600, dtype=dtype)
    c.pool.copy_(torch.randn(c.pool.shape, generator=g, device="cuda"))
    p = 60 * page
    dspark.cache_reserve(c, ints([p]), 0, seq=ints([0]))
    dspark.cache_fork(c, ints([0]), ints([1]), ints([p]))
    length = [p + 20 * page + 3, p + 11 * page, 33 * page + 1]
    dspark.cache_reserve(c, ints(length), 16)
    return c, length, [0, 2, 3], [p, 0], g


# bytes of a page's bounds are 4 kv D (bfloat16) or 8 kv D: 4.4 GB of them
@pytest.mark.parametrize("dtype,page,D,kv,pages", [(BF, 2, 128, 8, 1_080_000), (BF, 8, 64, 16, 1_080_000),
                                                   (F32, 1, 128, 8, 540_000)])
def test_far_pages_and_bounds(cuda, dtype, page, D, kv, pages):
    """The same sequences in the last pages of a large pool: the same results."""
    c, length, start, prefix, g = small_cache(dtype, page, D, kv, D)
    q = torch.randn(3, 4, 2 * kv, D, generator=g, device="cuda").to(dtype)
    want = calls(c, length, start, prefix, q, 9)
    far = pages - c.num_pages
    assert far * 2 * D * kv * q.element_size() > 1 << 32
    pool = torch.empty(1, 2, pages, kv, page, D, dtype=dtype, device="cuda")
    pool[:, :, far:] = c.pool
    table = torch.where(c.block_table >= 0, c.block_table + far, c.block_table)
    big = dspark.PagedCache.from_tensors(pool, table, c.page_count.clone(), ints([0]).expand(pages).contiguous(),
                                         torch.arange(pages, dtype=torch.int32, device="cuda"), c.control.clone())
    got = calls(big, length, start, prefix, q, 9)
    assert torch.equal(got[0][:, far:], want[0])
    for i, (x, y) in enumerate(zip(got[1:], want[1:])):
        assert torch.equal(x, y), i


@pytest.mark.parametrize("dtype,D", [(BF, 128), (BF, 64), (F32, 64)])
def test_smaller_calls_in_a_larger_ones_workspace(cuda, dtype, D):
    """Workspaces that hold what a larger call left, and whatever was there."""
    c, length, start, prefix, g = small_cache(dtype, 8, D, 4, D + 1)
    ws = dict(select=dspark.SelectWorkspace(c, 9, 16), sparse=dspark.SparseWorkspace(c, 9, 16, 16, 50),
              prefix=dspark.PrefixWorkspace(9, 16, 16, 4, D))
    for x in ws.values():
        x.buffer.fill_(255)  # NaN as floating-point numbers, -1 as whole ones
    for n, T, count in ((3, 16, 40), (3, 1, 5), (1, 3, 2), (2, 16, 50), (3, 2, 9)):
        q = torch.randn(n, T, 16, D, generator=g, device="cuda").to(dtype)
        a = (c, length[:n], start if n == 3 else [0, n], prefix if n == 3 else prefix[:1], q, count)
        for x, y in zip(calls(*a, ws), calls(*a)):
            assert torch.equal(x, y), (n, T, count)


def test_equal_rows_are_equal(cuda):
    """The same sequence more than once in a call, as a batch may have it."""
    c, length, _, _, g = small_cache(BF, 16, 128, 2, 5)
    q = torch.randn(1, 3, 8, 128, generator=g, device="cuda").to(BF).expand(4, -1, -1, -1).contiguous()
    seq, n = ints([1] * 4), ints([length[1]] * 4)
    bounds = dspark.cache_bounds(c, ints([0] * 4), n, seq=seq)
    pages = dspark.select_pages(c, 0, bounds, q, n, 6, seq=seq)
    assert (pages == pages[:1]).all()
    out, lse = dspark.sparse_attention(c, 0, q, n, pages, seq=seq, with_lse=True)
    whole = dspark.tree_attention(c, 0, q, n, seq=seq, with_lse=True)
    shared = dspark.prefix_attention(c, 0, q, n, ints([0, 4]), ints([500]), seq=seq, with_lse=True)
    # Rows are split between blocks alike or not, so weights have other references: each
    # is rounded to 2^-8 anew and so is the result; sums of fewer than 2048 float32
    # weights, each off by 2^-20 (of 2^x) and 2^-20 (of x, below 16), in another order.
    assert ((out - out[:1]).float().abs() <= 2.0 ** -7 * (c.pool.float().abs().max() + 1)).all()
    for x in (lse - lse[:1], shared[1] - whole[1]):
        assert (x.abs() <= 2 * (2.0 ** -19 + 2048 * 2.0 ** -24)).all()
    assert dspark.read_device_error(c) == 0
    assert math.isfinite(float(lse.sum()))


def test_more_pages_than_are_counted(cuda):
    """One sequence in 1024 rows of a call: 2^31 pages together; and in one."""
    wide = (1 << 21) + 1
    c = dspark.PagedCache(1, 2, 1, 1, 8, 1, wide, dtype=F32)
    c.pool.copy_(torch.arange(32.0, device="cuda").reshape(c.pool.shape))
    c.block_table.fill_(1)
    c.page_count.fill_(wide)
    start, length = ints([0]).repeat(1024), ints([1 << 21]).repeat(1024)
    seq = torch.zeros_like(start)
    bounds = torch.zeros(1, 2, 1, 2, 8, device="cuda")
    dspark.cache_bounds(c, start, length, bounds=bounds, seq=seq)
    assert dspark.read_device_error(c) == 7 and not bounds.any()
    start[1:] = 1 << 21  # the first alone
    dspark.cache_bounds(c, start, length, bounds=bounds, seq=seq)
    assert dspark.read_device_error(c) == 0
    assert torch.equal(bounds[0, 1, 0], c.pool[0, 0, 1, 0].expand(2, -1)) and not bounds[0, 0].any()


@pytest.mark.parametrize("dtype,D,kv", [(BF, 128, 2), (BF, 96, 2), (F32, 64, 2)])
def test_equal_rows_are_right(cuda, dtype, D, kv):
    """The same: each row's results against 64 bits, over selected pages, behind a
    prefix and over all."""
    c, length, _, _, g = small_cache(dtype, 16, D, kv, D)
    T, heads, count = 3, 4 * kv, 6
    q = torch.randn(1, T, heads, D, generator=g, device="cuda").to(dtype).expand(4, -1, -1, -1).contiguous()
    m = length[1]
    seq, n = ints([1] * 4), ints([m] * 4)
    bounds = dspark.cache_bounds(c, ints([0] * 4), n, seq=seq)
    pages = dspark.select_pages(c, 0, bounds, q, n, count, seq=seq)
    assert (pages == pages[:1]).all()
    results = {"sparse": dspark.sparse_attention(c, 0, q, n, pages, seq=seq, with_lse=True),
               "whole": dspark.tree_attention(c, 0, q, n, seq=seq, with_lse=True),
               "shared": dspark.prefix_attention(c, 0, q, n, ints([0, 4]), ints([500]), seq=seq, with_lse=True)}
    ids, slots = place(c, 1, m + T)
    k, v = (c.pool[0, i][ids.cuda(), :, slots.cuda()].transpose(0, 1) for i in (0, 1))
    sees = tree_sees(m, T, [(2 << t) - 1 for t in range(T)], 0, [0] * T)
    some = sees[None].repeat(kv, 1, 1)
    named = torch.zeros(kv, T, m // 16 + 1, dtype=torch.bool)
    named.scatter_(2, pages[0].cpu().long().transpose(0, 1), True)
    some[:, :, :m // 16 * 16] = named[:, :, :-1].repeat_interleave(16, dim=2)
    for name, (out, lse) in results.items():
        ro, rl, size, reach = attend_all(k, v, q[0], (some[:, None] if name == "sparse" else sees).cuda(), 1 / math.sqrt(D))
        bo, bl = attend_bounds(size, reach, ro, rl, m + T, D, dtype == BF)
        for b in range(4):
            assert ((out[b].double() - ro).abs() <= bo).all(), (name, b)
            assert ((lse[b].double() - rl).abs() <= bl).all(), (name, b)
    assert dspark.read_device_error(c) == 0
