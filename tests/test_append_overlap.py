"""The queries that cache_append writes must not lie over the rows it reads,
but where they are q itself."""
import ctypes

import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.test_cache_abi import FAKE, INVALID, append, lib  # noqa: F401  (a fixture)

FAR = FAKE + (1 << 30)
# 4 tokens, 4 query heads and 2 key heads of 64 dims, bfloat16: rows of 512 and
# 256 bytes, 512 and 256 bytes apart unless said otherwise; q_out has 2048 bytes
APART = dict(q=FAR, k=FAR + 8192, v=FAR + 16384, out=FAKE)


@pytest.mark.parametrize("over", [
    dict(q=FAKE + 16), dict(q=FAKE - 16), dict(q=FAKE + 2048 - 16), dict(q=FAKE - 2048 + 16),
    dict(k=FAKE), dict(k=FAKE + 2048 - 16), dict(k=FAKE - 1024 + 16), dict(k=FAKE + 512),
    dict(v=FAKE), dict(v=FAKE + 2048 - 16), dict(v=FAKE - 1024 + 16),
    dict(q=FAKE, k=FAKE + 1024),                     # in place, but over the keys
    dict(k=FAKE - 3 * 65536, ks=32768),              # the last row alone
    dict(v=FAKE - 65536 - 240, vs=32768),            # the second row's end
    dict(q=FAKE - 2 * 65536 - 496, qs=32768),
    dict(k=FAKE - 64 * (1 << 40) + 2032, ks=(1 << 40) * 32),
])
def test_overlaps_are_refused(lib, over):  # noqa: F811
    assert append(lib, **{**APART, **over}) == INVALID


def test_strides_past_64_bits_of_bytes(lib):  # noqa: F811
    """A row a quarter of the address space away does not wrap onto q_out."""
    assert append(lib, **{**APART, "k": FAKE, "ks": (1 << 62)}) == INVALID  # its first row


@pytest.mark.gpu
def test_rows_beside_each_other_are_taken(cuda):
    """q, k and v as parts of one projection's output, and q_out dense between
    their tokens: nothing that is read is written."""
    B, T, heads, kv, D = 1, 2, 4, 2, 64
    c = dspark.PagedCache(1, 4, 16, kv, D, 1, 4)
    length = torch.zeros(1, dtype=torch.int32, device="cuda")
    dspark.cache_reserve(c, length, T)
    g = torch.Generator(device="cuda").manual_seed(0)
    buf = torch.randn(B, T, 4096, generator=g, device="cuda").bfloat16()
    q = buf[:, :, :256].unflatten(2, (heads, D))
    k = buf[:, :, 256:384].unflatten(2, (kv, D))
    v = buf[:, :, 384:512].unflatten(2, (kv, D))
    a = dict(position=torch.arange(2, dtype=torch.int32, device="cuda")[None],
             cos_sin=torch.randn(2, D, generator=g, device="cuda"))
    want = dspark.cache_append(c, 0, q, k, v, length, **a)
    inside = buf[0, 0, 512:1024].view(B, T, heads, D)
    assert torch.equal(dspark.cache_append(c, 0, q, k, v, length, q_out=inside, **a), want)
    dense = q.contiguous()
    assert torch.equal(dspark.cache_append(c, 0, dense, k, v, length, q_out=dense, **a), want)
    for at in (504, 4096 - 16, 4096 - 512 + 8):  # over v's first row, over the second token
        over = buf.view(-1)[at:at + 512].view(B, T, heads, D)
        with pytest.raises(dspark.DsparkError):
            dspark.cache_append(c, 0, q, k, v, length, q_out=over, **a)
    assert dspark.read_device_error(c) == 0
