"""Blocks that work through many tiles: units of several tiles one after the
other in every block, whole and cut, with the running maximum raised from tile
to tile, windows, and NaN and infinities in places that some rows see and
others do not.  Units of at most 32 rows, of at most 128 and of more on the
tensor cores, and the float32 kernel's variants, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.cache_ref import place
from tests.test_gpu_tree_units import Units

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32
# dtype, head_dim, heads of a key head, tokens
FORMS = [(BF, 128, 4, 8), (BF, 64, 8, 1), (BF, 128, 8, 6), (BF, 64, 8, 6), (BF, 128, 3, 64), (BF, 64, 5, 40),
         (F32, 128, 4, 2), (F32, 64, 8, 6), (F32, 256, 1, 3), (BF, 96, 2, 7)]


def lengths(seed, n, low, high):
    return [int(x) for x in np.random.default_rng(seed).integers(low, high, n)]


def tiles(s):
    """Tiles of the call on the tensor cores (the float32 kernel has more)."""
    rows = 128 // (s.heads // s.kv)
    rows = rows if s.T <= rows else 2 * rows
    return sum(-(-c // rows) * s.kv * -(-(n + c) // 128) for n, c in zip(s.length, s.count))


def scale_keys(s, ramp):
    """Multiplies the keys of each sequence by ramp(tokens)."""
    for b, q in enumerate(s.seq):
        k = (s.k[b].float() * ramp(s.k[b].shape[1])[None, :, None]).to(s.c.dtype)
        ids, slots = place(s.c, q, k.shape[1])
        s.c.pool[s.layer, 0][ids.cuda(), :, slots.cuda()] = k.transpose(0, 1).cuda()
        s.k[b] = k


@pytest.mark.parametrize("dtype,D,group,T", FORMS)
@pytest.mark.parametrize("page,mask,low,high", [(64, "causal", 250, 2500), (16, "tree", 380, 390), (128, "holes", 1, 900)])
def test_many_tiles_a_block(cuda, dtype, D, group, T, page, mask, low, high):
    """Units of 2 to 20 tiles; of four tiles each; of 1 to 8."""
    kv = 8
    n = lengths(D + low, 36, low, high)
    count = [1 + (i * 7) % T for i in range(36)]
    s = Units(dtype, D, kv, group, T, n, page, mask, count=count, seq=list(range(40, 4, -1)), seed=T)
    assert tiles(s) > 6 * 152
    out, lse = torch.zeros_like(s.q), torch.zeros(36, T, kv * group, device="cuda")
    s.run(out=out, lse=lse)
    s.check(out, lse)
    again, again_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for _ in range(5):
        s.run(out=again, lse=again_lse)
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


@pytest.mark.parametrize("dtype,D,group,T", FORMS)
def test_one_sequence_over_all_blocks(cuda, dtype, D, group, T):
    """Each block has several tiles of one unit, and the ends of two."""
    s = Units(dtype, D, 2, group, T, [61000], 64, "causal", seed=T, layers=1)
    assert tiles(s) > 6 * 152
    s.check(*s.run())


@pytest.mark.parametrize("dtype,D,group,T", FORMS)
@pytest.mark.parametrize("window", [100, 700])
def test_windows_over_many_tiles(cuda, dtype, D, group, T, window):
    s = Units(dtype, D, 8, group, T, lengths(D + window, 60, 1, 2000), 32, "tree", window=window, seed=T)
    assert tiles(s) > 6 * 152
    s.check(*s.run())


@pytest.mark.parametrize("dtype,D,group,T", FORMS)
@pytest.mark.parametrize("size,scale", [(2.0, None), (8.0, None), (60.0, None), (-60.0, None), (60.0, -0.1)])
def test_the_maximum_rises_from_tile_to_tile(cuda, dtype, D, group, T, size, scale):
    """Scores that grow along the keys, by less than a weight may exceed one
    and by far more, and (size < 0) fall."""
    s = Units(dtype, D, 8, group, T, lengths(D, 16, 600, 1700), 64, "causal", seed=T)
    assert tiles(s) > 6 * 152
    scale_keys(s, lambda n: torch.linspace(0.05, 1.0, n).flip(0) * -size if size < 0 else torch.linspace(0.05, 1.0, n) * size)
    s.check(*(s.run() if scale is None else s.run(scale=scale)), scale=scale)


@pytest.mark.parametrize("dtype,D,group,T", [f for f in FORMS if f[3] > 1])
@pytest.mark.parametrize("low,high", [(130, 250), (260, 700)])
def test_special_values_reach_the_rows_that_see_them(cuda, dtype, D, group, T, low, high):
    """Values of drafted tokens that are NaN or infinite, in the second tile
    of many units: rows that see them have them, the others their own bits."""
    kv = 8
    s = Units(dtype, D, kv, group, T, lengths(D + T + low, 60, low, high), 16, "tree", seed=T + 1)
    assert tiles(s) > 4 * 152
    clean = s.run()[0]
    s.check(*s.run())
    spots = {0: float("inf"), T // 2: float("nan"), T - 1: -float("inf")}
    for b in range(s.B):
        ids, slots = place(s.c, b, s.length[b] + T)
        for i, (j, bad) in enumerate(spots.items()):
            s.c.pool[s.layer, 1, ids[s.length[b] + j], :, slots[s.length[b] + j], 3 + 20 * i] = bad
    out, lse = s.run()
    for b in range(s.B):
        left = torch.ones(T, kv * group, D, dtype=torch.bool, device="cuda")
        for i, (j, bad) in enumerate(spots.items()):
            sees = torch.tensor([bool((w >> j) & 1) for w in s.words[b]], device="cuda")
            x = out[b, sees, :, 3 + 20 * i].float()
            assert (torch.isnan(x) if math.isnan(bad) else x == bad).all()
            left[sees, :, 3 + 20 * i] = False
        assert torch.equal(out[b][left], clean[b][left])
    assert torch.equal(lse, s.run()[1]) and dspark.read_device_error(s.c) == 0


@pytest.mark.parametrize("dtype,D,group,T", [f for f in FORMS if f[3] > 1])
def test_special_values_at_a_windows_edge(cuda, dtype, D, group, T):
    """Infinite values of the committed token that all but the first drafted
    one have left behind, NaN before it, in many units."""
    kv, window = 8, 300
    n = lengths(D + T, 60, 500, 900)
    s = Units(dtype, D, kv, group, T, n, 16, "causal", window=window, seed=T + 2)
    s.position = [[x + t for t in range(T)] for x in n]
    s.check(*s.run())
    clean = s.run()[0]
    for b in range(s.B):
        ids, slots = place(s.c, b, n[b])
        edge = n[b] - window + 1
        s.c.pool[s.layer, 1, ids[edge], :, slots[edge], 5] = float("inf")
        s.c.pool[s.layer][:, ids[edge - 100:edge].cuda(), :, slots[edge - 100:edge].cuda()] = float("nan")
    out = s.run()[0]
    assert (out[:, 0, :, 5] == float("inf")).all() and torch.equal(out[:, 1:], clean[:, 1:])
    keep = [d for d in range(D) if d != 5]
    assert torch.equal(out[:, 0][..., keep], clean[:, 0][..., keep])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 3])
def test_a_window_below_the_tokens_leaves_them_to_the_mask(cuda, dtype, window):
    """A window rules the committed tokens alone: without a mask a token sees
    all drafted ones up to itself, those beyond the window too."""
    s = Units(dtype, 64, 2, 4, 9, [0, 1, 50, 130], 16, "causal", window=window, seed=window)
    s.check(*s.run(mask=None, position=None))
    narrow = [((2 << t) - 1) & ~((1 << max(0, t - window + 1)) - 1) for t in range(9)]
    s.words = [narrow] * 4  # the caller's own words make it slide over them too
    s.check(*s.run(mask=torch.tensor(narrow, device="cuda"), position=None))
