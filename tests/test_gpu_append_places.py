"""What cache_append leaves alone: places that no page holds, tokens behind a
sequence's count, other sequences, layers and pages."""
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.test_gpu_cache import error, ints, make

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


@pytest.mark.parametrize("dtype,dim,rot", [(BF, 64, 64), (BF, 128, 128), (F32, 64, 64), (BF, 40, 12), (F32, 24, 24)])
def test_only_held_places_are_written(cuda, dtype, dim, rot):
    c, _ = make(page=16, num_pages=20, kv_heads=1, dim=dim, layers=2, dtype=dtype)
    dspark.cache_reserve(c, ints([0, 0]), 16)
    g = torch.Generator(device="cuda").manual_seed(dim)
    q = torch.randn(2, 2, 2, dim, generator=g, device="cuda").to(dtype)
    k = torch.randn(2, 2, 1, dim, generator=g, device="cuda").to(dtype)
    v = torch.randn(2, 2, 1, dim, generator=g, device="cuda").to(dtype)
    a = dict(position=ints([[0, 1], [2, 3]]), cos_sin=torch.randn(8, rot, generator=g, device="cuda"))
    before = c.pool.clone()
    queries = None
    for nowhere in ([16, 40], [-1, -2147483648], [-2147483648, 2147483647], [2147483646, 1 << 30], [17, -2]):
        got = dspark.cache_append(c, 1, q, k, v, ints(nowhere), **a)
        assert error(c) == 7 and torch.equal(before, c.pool)
        queries = got if queries is None else queries
        assert torch.equal(got, queries)
    # place 15 is the last one held: the first token of the second sequence
    page = int(c.block_table[1, 0])
    assert torch.equal(dspark.cache_append(c, 1, q, k, v, ints([2147483646, 15]), **a), queries)
    assert error(c) == 7
    changed = (c.pool != before).any(dim=-1).nonzero().tolist()
    assert changed == [[1, plane, page, 0, 15] for plane in (0, 1)]
    assert torch.equal(c.pool[1, 1, page, 0, 15], v[1, 0, 0])
    # the same keys as where both tokens have places
    key = c.pool[1, 0, page, 0, 15].clone()
    dspark.cache_append(c, 0, q, k, v, ints([0, 0]), **a)
    assert error(c) == 0 and torch.equal(c.pool[0, 0, page, 0, 0], key)
    assert torch.equal(c.pool[0, 1, page, 0, :2], v[1, :, 0])
    first = int(c.block_table[0, 0])
    changed = (c.pool[0] != before[0]).any(dim=-1).nonzero().tolist()
    assert changed == [[plane, p, 0, i] for plane in (0, 1) for p in sorted((page, first)) for i in (0, 1)]
