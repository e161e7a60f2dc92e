"""Many units a block: calls whose tiles are several times the GPU's
multiprocessors, so that every block works through units of several tiles one
after the other, whole ones and ones that its share cuts.  Units of at most 32
rows, of at most 128 and of more, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.cache_ref import attend_bounds, place, tree_sees
from tests.test_gpu_tree_attention import Case, ints

pytestmark = pytest.mark.gpu
BF = torch.bfloat16


def attend_all(k, v, q, sees, scale):
    """cache_ref.attend for all rows of a sequence at once, on the GPU."""
    t, heads, D = q.shape
    kv, n, _ = k.shape
    K, V = k.double(), v.double()
    Q = q.double().reshape(t, kv, heads // kv, D).permute(1, 2, 0, 3)     # [kv, group, t, D]
    z = (Q @ K[:, None].transpose(2, 3)) * scale                          # [kv, group, t, n]
    z = z.masked_fill(~sees, -math.inf)
    m = z.amax(dim=-1, keepdim=True)
    p = torch.exp(z - torch.where(torch.isinf(m), 0.0, m))
    total = p.sum(dim=-1, keepdim=True)
    some = torch.where(total > 0, total, 1.0)
    out, size = (p @ V[:, None]) / some, (p @ V[:, None].abs()) / some
    lse = (m + torch.log(total)).squeeze(-1)
    reach = (Q.abs() @ K[:, None].transpose(2, 3).abs()).masked_fill(~sees, 0.0).amax(dim=-1) * abs(scale)

    def rows(x):
        return x.movedim(2, 0).reshape(t, heads, *x.shape[3:])
    return rows(out), rows(lse), rows(size), rows(reach)


class Units(Case):
    def check(self, out, lse, scale=None):
        scale = scale or 1.0 / math.sqrt(self.D)
        out, lse = out.double(), lse.double()
        for b in range(self.B):
            t = self.count[b]
            if not t:
                continue
            sees = tree_sees(self.length[b], t, self.words[b], self.window, self.position[b]).cuda()
            ro, rl, size, reach = attend_all(self.k[b].cuda(), self.v[b].cuda(), self.q[b, :t], sees, scale)
            bo, bl = attend_bounds(size, reach, ro, rl, sees.shape[1], self.D, self.c.dtype == BF)
            none = torch.isinf(rl)
            assert torch.equal(torch.isinf(lse[b, :t]), none), b
            assert (out[b, :t][none] == 0).all(), b
            assert ((out[b, :t] - ro).abs() <= bo).all(), (b, ((out[b, :t] - ro).abs() / bo).max())
            assert ((lse[b, :t] - rl).abs()[~none] <= bl[~none]).all(), b
        assert dspark.read_device_error(self.c) == 0


# head_dim, key heads, heads of each, tokens: 8, 48 and 192 rows
FORMS = [(128, 8, 1, 8), (64, 8, 1, 8), (128, 8, 8, 6), (64, 8, 8, 6), (128, 8, 3, 64), (64, 8, 3, 64)]


@pytest.mark.parametrize("D,kv,group,T", FORMS)
@pytest.mark.parametrize("lengths", [(120, 250), (200, 201), (1, 400)])
def test_what_lies_behind_the_sequences_stays_there(cuda, D, kv, group, T, lengths):
    """NaN in every place behind a sequence's end, units of one to four tiles
    that follow one another in each block, and where units have more than 128
    rows smaller ones before them: the results are those of the same call with
    zeros there, bit for bit, and those of 64 bits."""
    rng = np.random.default_rng(D + T + lengths[0])
    length = [int(x) for x in rng.integers(*lengths, 88)]
    count = [int(x) for x in rng.integers(1, T + 1, 88)]
    if T == 64 and lengths[0] == 200:  # joined units of 60 rows, then one tile of 192 rows
        for b in range(0, 88, 2):
            length[b], count[b], length[b + 1], count[b + 1] = 150 + b, 20, b // 2, 64
    s = Units(BF, D, kv, group, T, length, 16, "causal", count=count, seed=D)
    out, lse = torch.zeros_like(s.q), torch.zeros(88, T, kv * group, device="cuda")
    s.run(out=out, lse=lse)
    s.check(out, lse)
    again, again_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for _ in range(10):
        s.run(out=again, lse=again_lse)
        assert torch.equal(out, again) and torch.equal(lse, again_lse)
    s.c.pool.nan_to_num_(0.0)
    s.run(out=again, lse=again_lse)
    assert torch.equal(out, again) and torch.equal(lse, again_lse)
