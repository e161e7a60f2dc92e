"""Attention of sequences that share prefixes, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.cache_ref import as_int64, attend_bounds, place, tree_sees, tree_words
from tests.test_gpu_tree_units import attend_all

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Prefix:
    """Groups (prefix tokens, members' own tokens): the members are forks of a
    sequence that holds the prefix.  NaN in every place that holds no token."""

    def __init__(self, dtype, D, kv, group, T, groups, page, mask="causal", count=None, seed=0, alone=()):
        rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.T, self.D, self.kv, self.heads, self.layer = T, D, kv, kv * group, 1
        sizes = [len(m) for _, m in groups]
        self.B = B = sum(sizes) + len(alone)
        self.count = count or [T] * B
        self.length = [p + n for p, m in groups for n in m] + list(alone)
        total = sum(-(-(n + T) // page) + 1 for n in self.length) + 5
        widest = max(-(-(n + T) // page) for n in self.length) + 2
        self.c = c = dspark.PagedCache(2, total, page, kv, D, B + 1, widest, dtype=dtype)
        c.free_list.copy_(torch.randperm(total, generator=g, device="cuda").int())
        c.pool.fill_(math.nan)
        self.seq = [B - i for i in range(B)]  # row i of a call is sequence B - i
        at = 0
        for p, m in groups:
            if m:
                lead = self.seq[at]
                dspark.cache_reserve(c, ints([p]), 0, seq=ints([lead]))
                self.write(lead, 0, p, g)
                for s in self.seq[at + 1:at + len(m)]:
                    dspark.cache_fork(c, ints([lead]), ints([s]), ints([p]))
            at += len(m)
        dspark.cache_reserve(c, ints(self.length), T, seq=ints(self.seq))
        at = 0
        for p, m in groups + [(0, alone)]:
            for i in range(len(m)):
                self.write(self.seq[at + i], p, self.length[at + i] + self.count[at + i], g)
            at += len(m)
        self.group_start = np.cumsum([0] + sizes).tolist()
        self.prefix = [p for p, _ in groups]
        words = [tree_words(mask, T, rng) for _ in range(B)]
        self.words = [w for w, _ in words]
        self.mask = as_int64(self.words).cuda()
        self.q = torch.randn(B, T, self.heads, D, generator=g, device="cuda").to(dtype)

    def write(self, s, start, end, g):
        ids, slots = place(self.c, s, end)
        ids, slots = ids[start:].cuda(), slots[start:].cuda()
        for plane in range(2):
            for layer in range(2):
                self.c.pool[layer, plane][ids, :, slots] = torch.randn(
                    end - start, self.kv, self.D, generator=g, device="cuda").to(self.c.dtype)

    def run(self, **over):
        a = dict(mask=self.mask, token_count=ints(self.count), seq=ints(self.seq), with_lse=True)
        start, prefix = over.pop("group_start", self.group_start), over.pop("prefix", self.prefix)
        length = over.pop("length", self.length)
        a.update(over)
        return dspark.prefix_attention(self.c, self.layer, self.q, ints(length), ints(start), ints(prefix), **a)

    def check(self, out, lse, scale=None, error=0, rows=None):
        scale = scale or 1.0 / math.sqrt(self.D)
        for b in rows if rows is not None else range(self.B):
            t = self.count[b]
            if not t:
                continue
            ids, slots = place(self.c, self.seq[b], self.length[b] + t)
            k, v = (self.c.pool[self.layer, i][ids.cuda(), :, slots.cuda()].transpose(0, 1) for i in (0, 1))
            sees = tree_sees(self.length[b], t, self.words[b], 0, [0] * t).cuda()
            ro, rl, size, reach = attend_all(k, v, self.q[b, :t], sees, scale)
            bo, bl = attend_bounds(size, reach, ro, rl, sees.shape[1], self.D, self.c.dtype == BF)
            none = torch.isinf(rl)
            o, l = out[b, :t].double(), lse[b, :t].double()
            assert torch.equal(torch.isinf(l), none), b
            assert (o[none] == 0).all(), b
            assert ((o - ro).abs() <= bo).all(), (b, ((o - ro).abs() / bo).max())
            assert ((l - rl).abs()[~none] <= bl[~none]).all(), b
        assert dspark.read_device_error(self.c) == error


SHAPES = [  # dtype, D, kv, group, T, groups, page, mask
    (BF, 128, 2, 4, 1, [(960, [0, 40])], 64, "causal"),
    (BF, 128, 2, 4, 8, [(256, [0, 1, 100]), (64, [500])], 64, "causal"),
    (BF, 128, 1, 8, 61, [(320, [5, 0, 7]), (0, [9, 3]), (1000, [10, 300])], 32, "tree"),
    (BF, 64, 2, 5, 7, [(112, [30, 0]), (16, [3] * 9)], 16, "full"),
    (BF, 64, 4, 8, 1, [(512, list(range(0, 88)))], 16, "causal"),
    (BF, 64, 1, 32, 9, [(200, [0, 70, 3])], 64, "holes"),          # a prefix that ends inside a page
    (BF, 128, 2, 7, 19, [(129, [511, 0, 90]), (127, [1, 2])], 256, "holes"),
    (BF, 128, 1, 1, 2, [(3000, [1, 2, 3, 4])], 16, "causal"),
    (BF, 128, 1, 2, 1, [(7, [0, 0])], 8, "causal"),
    (BF, 96, 2, 3, 6, [(77, [0, 20]), (16, [1, 1])], 16, "tree"),   # dims of the next larger form
    (BF, 96, 1, 8, 61, [(320, [5, 0, 7]), (0, [9, 3]), (1000, [10, 300])], 32, "tree"),
    (BF, 80, 2, 4, 1, [(960, [0, 40])], 64, "causal"),
    (BF, 112, 2, 4, 8, [(256, [0, 1, 100]), (64, [500])], 64, "causal"),
    (BF, 48, 4, 8, 1, [(512, list(range(0, 88)))], 16, "causal"),
    (BF, 32, 2, 5, 7, [(112, [30, 0]), (16, [3] * 9)], 16, "full"),
    (BF, 16, 1, 32, 9, [(200, [0, 70, 3])], 64, "holes"),
    (BF, 72, 2, 3, 6, [(77, [0, 20]), (16, [1, 1])], 16, "tree"),   # FFMA: dim
    (BF, 128, 1, 4, 5, [(48, [50, 1, 0])], 12, "tree"),             # FFMA: page
    (BF, 256, 1, 2, 4, [(65, [0, 64])], 32, "causal"),
    (BF, 8, 1, 2, 3, [(10, [1, 2]), (33, [200])], 16, "tree"),
    (F32, 64, 2, 3, 7, [(777, [0, 64, 1])], 16, "full"),
    (F32, 128, 1, 8, 33, [(190, [5, 5])], 64, "tree"),
    (F32, 128, 2, 1, 1, [(63, [0, 1]), (64, [0, 1]), (65, [2, 0])], 7, "causal"),
    (F32, 256, 1, 2, 6, [(100, [1, 30])], 16, "holes"),
    (F32, 40, 1, 32, 3, [(70, [0, 0])], 1, "causal"),
]


@pytest.mark.parametrize("dtype,D,kv,group,T,groups,page,mask", SHAPES)
def test_matches_64_bits(cuda, dtype, D, kv, group, T, groups, page, mask):
    s = Prefix(dtype, D, kv, group, T, groups, page, mask, seed=T + D, alone=(12, 0))
    got = s.run()
    s.check(*got)
    again = s.run()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_what_the_first_row_holds_is_read(cuda, dtype):
    """The other rows' table entries of the prefix are not looked at."""
    s = Prefix(dtype, 64, 2, 2, 4, [(96, [3, 20, 7]), (32, [1, 1])], 32, seed=1)
    want = s.run()
    for row, n in ((1, 3), (2, 3), (4, 1)):
        s.c.block_table[s.seq[row], :n] = 1 << 30
    got = s.run()
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert dspark.read_device_error(s.c) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padding(cuda, dtype):
    """Fewer tokens than T and none at all, of a group's first row too: rows
    behind the last token stay as they were; empty groups."""
    count = [0, 8, 3, 1, 8, 0, 5]
    s = Prefix(dtype, 64, 2, 4, 8, [(100, [5, 0, 9]), (0, []), (40, [2, 2]), (64, [1])], 16, count=count, alone=(30,))
    s.q[0] = math.nan  # rows that are not there may hold anything
    out = torch.full((7, 8, 8, 64), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((7, 8, 8), 6.0, device="cuda")
    got = s.run(out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    s.check(out, lse)
    for b, n in enumerate(count):
        assert (out[b, n:] == 5).all() and (lse[b, n:] == 6).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scales_and_masks(cuda, dtype):
    s = Prefix(dtype, 128, 1, 2, 12, [(100, [5, 0, 9]), (40, [2, 2])], 16, "holes")
    s.check(*s.run(scale=0.3), scale=0.3)
    s.check(*s.run(scale=-0.05), scale=-0.05)
    s.words = [[(2 << t) - 1 for t in range(12)]] * 5
    s.check(*s.run(mask=None))
    s.check(*s.run(mask=as_int64(s.words[0]).cuda()))
    a, none = s.run(mask=None, with_lse=False)
    assert none is None and torch.equal(a, s.run(mask=None)[0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_special_values(cuda, dtype):
    """A NaN among a sequence's own tokens stays its own; one in the prefix
    reaches the whole group and nobody else."""
    s = Prefix(dtype, 64, 1, 2, 5, [(100, [5, 40, 9]), (40, [2, 2])], 16)
    clean = s.run()
    ids, slots = place(s.c, s.seq[1], 120)
    s.c.pool[1, 1, ids[110], 0, slots[110], 7] = math.inf
    got = s.run()
    assert torch.isinf(got[0][1, :, :, 7]).all() and torch.equal(got[1], clean[1])
    rest = [0, 2, 3, 4]
    assert torch.equal(got[0][rest], clean[0][rest])
    s.c.pool[1, 1, ids[50], 0, slots[50], 9] = math.nan
    got = s.run()
    assert torch.isnan(got[0][:3, :, :, 9]).all() and torch.equal(got[0][3:], clean[0][3:])


# heads of each key head, tokens, members: units of few, 128 and 256 rows
@pytest.mark.parametrize("D,kv,group,T,members", [(128, 8, 1, 8, 4), (64, 8, 1, 8, 4), (128, 8, 8, 6, 11), (64, 8, 8, 6, 11),
                                                  (128, 2, 4, 32, 8), (64, 2, 4, 33, 8), (64, 8, 4, 1, 44),
                                                  (96, 8, 1, 8, 4), (48, 8, 8, 6, 11), (80, 2, 4, 32, 8)])
def test_units_that_follow_one_another(cuda, D, kv, group, T, members):
    """Prefixes and suffixes of one to several tiles behind one another in each
    block, with NaN in every place that holds no token."""
    rng = np.random.default_rng(D + T)
    groups = [(int(rng.integers(1, 900)), [int(x) for x in rng.integers(0, 300, members)]) for _ in range(88 // members)]
    n = sum(len(m) for _, m in groups)
    count = [int(x) for x in rng.integers(1, T + 1, n)]
    s = Prefix(BF, D, kv, group, T, groups, 16, count=count, seed=D)
    out, lse = torch.zeros_like(s.q), torch.zeros(n, T, kv * group, device="cuda")
    s.run(out=out, lse=lse)
    s.check(out, lse)
    again, again_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for _ in range(5):
        s.run(out=again, lse=again_lse)
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_groups_that_are_none(cuda, dtype):
    """Each sequence is attended by itself, and the error word says so."""
    s = Prefix(dtype, 64, 1, 2, 4, [(100, [5, 40, 9]), (48, [2, 2])], 16, alone=(7,))
    s.check(*s.run(group_start=[0, 3, 5]))
    for start in ([0, 3, 7], [-1, 3, 5], [0, 5, 3], [3, 0, 5], [0, 2147483647, 5]):
        s.check(*s.run(group_start=start), error=12)
    s.check(*s.run(prefix=[-1, 48]), error=12)
    s.check(*s.run(prefix=[2147483647, 48]), error=12)   # the first row does not hold it
    s.check(*s.run(prefix=[200, 48]), error=12)
    s.check(*s.run(prefix=[108, 48]), error=12, rows=[0, 3, 4, 5])   # row 0 has fewer
    s.check(*s.run(group_start=[0, 1], prefix=[100]))
    s.check(*s.run(group_start=[0, 0], prefix=[100]))
    s.check(*s.run(group_start=[3, 5], prefix=[33]))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_first_row_that_has_less_than_the_prefix(cuda, dtype):
    """What its pages hold behind its own tokens is not read by the others."""
    s = Prefix(dtype, 64, 1, 2, 4, [(100, [5, 40, 9]), (48, [2, 2])], 16, alone=(7,))
    s.check(*s.run(prefix=[108, 48]), error=12)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sequences_out_of_range_are_left(cuda, dtype):
    s = Prefix(dtype, 64, 1, 2, 4, [(48, [5, 40, 9])], 16, alone=(7,))
    good = s.run()
    for over, code, row in ((dict(seq=ints([4, 9, 2, 1])), 6, 1), (dict(seq=ints([4, 3, -1, 1])), 6, 2),
                            (dict(length=[53, 88, 1000, 7]), 7, 2), (dict(length=[53, -1, 57, 7]), 7, 1)):
        out, lse = torch.full_like(s.q, 3.0), torch.full((4, 4, 2), 3.0, device="cuda")
        s.run(out=out, lse=lse, **over)
        assert dspark.read_device_error(s.c) == code
        assert (out[row] == 3).all() and (lse[row] == 3).all()
        rest = [b for b in range(4) if b != row]
        s.check(out, lse, rows=rest)
    # a first row that is none: the others are attended by themselves
    out = torch.full_like(s.q, 3.0)
    got = s.run(out=out, seq=ints([9, 3, 2, 1]))
    assert dspark.read_device_error(s.c) in (6, 12) and (out[0] == 3).all()
    s.check(*got, rows=[1, 2, 3])
    again = s.run()
    assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_graph_replay_and_streams(cuda, dtype):
    """A captured call reads groups, prefixes and lengths anew, and two graphs with
    workspaces of their own replay in any order; another stream."""
    s = Prefix(dtype, 128, 2, 2, 6, [(200, [3, 40, 0]), (48, [5, 5])], 16, "tree")
    length, start, prefix = ints(s.length), ints(s.group_start), ints(s.prefix)
    seq, count = ints(s.seq), ints(s.count)
    out = [torch.zeros_like(s.q) for _ in range(2)]
    lse = [torch.zeros(5, 6, 4, device="cuda") for _ in range(2)]
    ws = [dspark.PrefixWorkspace(9, 8, 4, 2, 128) for _ in range(2)]

    def call(i, **more):
        dspark.prefix_attention(s.c, s.layer, s.q, length, start, prefix, mask=s.mask, seq=seq, token_count=count,
                                out=out[i], lse=lse[i], workspace=ws[i], **more)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call(0)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            call(i)
    for new_start, new_prefix in (([0, 3, 5], [200, 48]), ([0, 2, 5], [120, 0]), ([0, 0, 3], [1, 200]), ([1, 3, 5], [64, 48])):
        start.copy_(ints(new_start))
        prefix.copy_(ints(new_prefix))
        for g in graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            s.check(out[i], lse[i])
    want = [out[0].clone(), lse[0].clone()]
    torch.cuda.synchronize()
    call(1, stream=stream)
    stream.synchronize()
    assert torch.equal(out[1], want[0]) and torch.equal(lse[1], want[1])


@pytest.mark.parametrize("D,group,T", [(128, 4, 2), (64, 8, 6), (64, 5, 40)])
def test_a_wait_that_runs_out_is_reported(cuda, monkeypatch, D, group, T):
    s = Prefix(BF, D, 4, group, T, [(700, [30, 0]), (300, [50, 200])], 16)
    a = dict(out=torch.zeros_like(s.q), lse=torch.zeros(4, T, 4 * group, device="cuda"),
             workspace=dspark.PrefixWorkspace(4, T, 4 * group, 4, D))
    s.run(**a)
    s.check(a["out"], a["lse"])
    want = [a["out"].clone(), a["lse"].clone()]
    monkeypatch.setenv("DSPARK_TEST_STALL_WAIT", "1")
    s.run(**a)
    torch.cuda.synchronize()
    assert dspark.read_device_error(s.c) == 2 and dspark.read_device_error(s.c) == 0
    monkeypatch.delenv("DSPARK_TEST_STALL_WAIT")
    s.run(**a)
    assert torch.equal(a["out"], want[0]) and torch.equal(a["lse"], want[1])
    assert dspark.read_device_error(s.c) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_prefix_that_the_only_row_does_not_have(cuda, dtype):
    """A group of one row says so too; an empty group's prefix is not looked at."""
    s = Prefix(dtype, 64, 1, 2, 4, [(100, [5]), (48, [2, 2])], 16, alone=(7,))
    s.check(*s.run())
    s.check(*s.run(prefix=[105, 48]))
    s.check(*s.run(prefix=[106, 48]), error=12)
    s.check(*s.run(prefix=[2147483647, 48]), error=12)
    s.check(*s.run(group_start=[0, 0, 0], prefix=[1000, 2147483647]))
    s.check(*s.run(group_start=[4, 4], prefix=[1000]))
