"""Special values, windows and large scores for units of few, more and many
rows: at most 32, at most 128 and more, which are treated differently."""
import math

import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.cache_ref import place
from tests.test_gpu_tree_attention import Case

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
FORMS = [(BF, 128, 5), (BF, 128, 8), (BF, 128, 32), (BF, 64, 5), (BF, 64, 8), (BF, 64, 32),
         (F32, 128, 8), (F32, 64, 32)]  # dtype, head_dim, heads of a key head, for 6 tokens


@pytest.mark.parametrize("dtype,D,group", FORMS)
def test_values_that_some_rows_see(cuda, dtype, D, group):
    s = Case(dtype, D, 1, group, 6, [300, 40, 0], 16, "tree", seed=5)
    clean = s.run()[0].float()
    spots = {3: float("nan"), 2: float("inf"), 4: -float("inf")}
    for b in range(3):
        ids, slots = place(s.c, b, s.length[b] + 6)
        for j, bad in spots.items():
            s.c.pool[s.layer, 1, ids[s.length[b] + j], 0, slots[s.length[b] + j], j] = bad
    out = s.run()[0].float()
    for b in range(3):
        for t in range(6):
            seen = [j for j in spots if (s.words[b][t] >> j) & 1]
            for j in seen:
                x = out[b, t, :, j]
                assert (torch.isnan(x) if math.isnan(spots[j]) else x == spots[j]).all()
            rest = [d for d in range(D) if d not in seen]
            assert torch.equal(out[b, t][:, rest], clean[b, t][:, rest])


@pytest.mark.parametrize("dtype,D,group", FORMS)
def test_keys_that_some_rows_see(cuda, dtype, D, group):
    s = Case(dtype, D, 1, group, 6, [200, 7], 16, "tree", seed=6)
    clean = s.run()[0].float()
    for b in range(2):
        ids, slots = place(s.c, b, s.length[b] + 6)
        s.c.pool[s.layer, 0, ids[s.length[b] + 3], 0, slots[s.length[b] + 3]] = float("nan")
    out = s.run()[0].float()
    for b in range(2):
        for t in range(6):
            if (s.words[b][t] >> 3) & 1:
                assert torch.isnan(out[b, t]).all()
            else:
                assert torch.equal(out[b, t], clean[b, t])


@pytest.mark.parametrize("dtype,D,group", FORMS)
def test_a_windows_edge(cuda, dtype, D, group):
    s = Case(dtype, D, 1, group, 6, [400, 60], 16, "causal", window=100, seed=7)
    s.check(*s.run())
    clean = s.run()[0].float()
    # position 400 + t sees tokens from 301 + t on: token 302 by t = 0, 1
    ids, slots = place(s.c, 0, 406)
    s.c.pool[s.layer, 1, ids[302], 0, slots[302], 5] = float("inf")
    s.c.pool[s.layer, 1, ids[250], 0, slots[250]] = float("nan")
    out = s.run()[0].float()
    assert (out[0, :2, :, 5] == float("inf")).all() and torch.equal(out[0, 2:], clean[0, 2:])
    keep = [d for d in range(D) if d != 5]
    assert torch.equal(out[0, :2][..., keep], clean[0, :2][..., keep])


@pytest.mark.parametrize("dtype,D,group", FORMS)
@pytest.mark.parametrize("size,scale", [(3.0, None), (3000.0, None), (30.0, -0.2)])
def test_scores_that_grow(cuda, dtype, D, group, size, scale):
    """Every tile raises the maximum, by little or past float32's exponents."""
    s = Case(dtype, D, 1, group, 6, [900], 64, "causal", seed=8)
    ramp = torch.linspace(0.1, 1.0, 906)[None, :, None] * size
    s.k = [(s.k[0].float() * ramp).to(dtype)]
    ids, slots = place(s.c, 0, 906)
    s.c.pool[s.layer, 0][ids.cuda(), :, slots.cuda()] = s.k[0].transpose(0, 1).cuda()
    s.check(*(s.run() if scale is None else s.run(scale=scale)), scale=scale)


@pytest.mark.parametrize("dtype,D,group", FORMS)
def test_units_over_several_blocks(cuda, dtype, D, group):
    s = Case(dtype, D, 1, group, 6, [9000, 1, 130], 64, "causal", seed=9)
    a, b = s.run(), s.run()
    s.check(*a)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype,D,group", [(BF, 128, 5), (BF, 64, 32), (F32, 64, 8)])
def test_nothing_to_do(cuda, dtype, D, group):
    """Counts of zero and below for all, and lengths of zero: nothing is
    written, or a token sees itself alone."""
    s = Case(dtype, D, 1, group, 6, [300, 40, 0], 16, "causal", seed=11)
    for none in (0, -1, -(2 ** 31)):
        out, lse = torch.full_like(s.q, 3.0), torch.full((3, 6, group), 3.0, device="cuda")
        s.count = [none] * 3
        s.run(out=out, lse=lse)
        assert (out == 3).all() and (lse == 3).all()
        dspark.read_device_error(s.c)
    s = Case(dtype, D, 1, group, 1, [0, 0], 16, "causal", seed=12)
    s.check(*s.run())
    assert torch.equal(s.run()[0][0, 0], s.v[0][0, 0].to("cuda").expand(group, D))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_counts_beyond_the_call(cuda, dtype):
    """A count above T is T."""
    s = Case(dtype, 64, 1, 2, 4, [30, 10, 60], 16, "causal", seed=13)
    good = s.run()[0]
    s.count = [4, 5, 2 ** 31 - 1]
    assert torch.equal(s.run()[0], good)
    assert dspark.read_device_error(s.c) == 0


WIDE_FFMA = [  # dtype, head_dim, key heads, group, tokens, lengths, page: the FFMA kernel, many rows
    (F32, 256, 1, 8, 5, [100, 33], 16), (BF, 256, 2, 32, 3, [70, 0], 24), (BF, 96, 1, 16, 4, [130], 12),
    (F32, 72, 1, 7, 9, [90, 1], 5), (F32, 8, 1, 32, 4, [77], 3), (F32, 128, 1, 25, 1, [200, 64], 16),
    (BF, 200, 1, 17, 2, [65], 7), (F32, 64, 2, 6, 64, [50], 16), (F32, 160, 1, 3, 9, [31, 32, 33], 32)]


@pytest.mark.parametrize("dtype,D,kv,group,T,length,page", WIDE_FFMA)
def test_many_rows_of_any_width(cuda, dtype, D, kv, group, T, length, page):
    s = Case(dtype, D, kv, group, T, length, page, "tree", seed=D + T)
    s.check(*s.run())
    s.window = 40
    s.check(*s.run())
