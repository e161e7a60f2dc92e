"""The bounds of pages and the pages that they select, against 64 bits."""
import math
import sys
import threading

import numpy as np
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.cache_ref import place
from tests.part_ref import choose, page_bounds, page_scores

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A cache of sequences with random keys, NaN in every other place."""

    def __init__(self, dtype, D, kv, group, T, length, page, layers=2, seq=None, count=None, seed=0, wide=0):
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.T, self.kv, self.D, self.page = len(length), T, kv, D, page
        self.length, self.layers = length, layers
        self.seq = seq or list(range(self.B))
        self.tokens = count or [T] * self.B
        total = sum(-(-n // page) for n in length) + 2
        most = max(max(-(-n // page) for n in length), 1) + wide
        self.c = dspark.PagedCache(layers, total, page, kv, D, max(self.seq) + 2, most, dtype=dtype)
        self.c.free_list.copy_(torch.randperm(total, generator=g, device="cuda").int())
        dspark.cache_reserve(self.c, ints(length), 0, seq=ints(self.seq))
        self.c.pool.fill_(float("nan"))
        self.keys = []  # of each sequence [layers, kv, n, D]
        for s, n in zip(self.seq, length):
            k = torch.randn(layers, kv, n, D, generator=g, device="cuda").to(dtype)
            ids, slots = place(self.c, s, n)
            if n:
                self.c.pool[:, 0][:, ids.cuda(), :, slots.cuda()] = k.permute(2, 0, 1, 3)
            self.keys.append(k)
        self.q = torch.randn(self.B, T, kv * group, D, generator=g, device="cuda").to(dtype)

    def bounds(self, start=None, **over):
        return dspark.cache_bounds(self.c, ints(start or [0] * self.B), ints(self.length), seq=ints(self.seq), **over)

    def check(self, bounds, pages, count, first=0, last=0, shared=False, layer=1, q=None):
        pages, q = pages.cpu(), (self.q if q is None else q).cpu()
        for b, s in enumerate(self.seq):
            F, t = self.length[b] // self.page, self.tokens[b]
            if not t:
                continue
            ids = self.c.block_table[s, :F].long()
            score = page_scores(q[b, :t], bounds[layer][ids].cpu())
            if shared:
                score = score.amax(dim=0, keepdim=True)
            for i in range(score.shape[0]):
                for h in range(self.kv):
                    want = choose(score[i, h].tolist(), count, first, last)
                    got = pages[b, i, h].tolist()
                    assert got == want + [-1] * (count - len(want)), (b, i, h)
        assert dspark.read_device_error(self.c) == 0


@pytest.mark.parametrize("dtype,D,page,length", [
    (BF, 128, 64, [0, 63, 64, 1000]), (BF, 64, 16, [500, 16]), (BF, 96, 12, [100]), (BF, 8, 1, [5, 0, 33]),
    (BF, 256, 32, [70]), (BF, 72, 7, [50, 7]), (F32, 64, 16, [77, 160]), (F32, 256, 8, [40]), (F32, 40, 3, [31]),
    (F32, 136, 128, [300]), (BF, 40, 256, [700])])
def test_bounds(cuda, dtype, D, page, length):
    s = Case(dtype, D, 3, 1, 1, length, page, seq=[2 * i for i in range(len(length))], seed=D)
    total = s.c.num_pages
    before = torch.full((2, total, 3, 2, D), 7.0, dtype=dtype, device="cuda")
    got = s.bounds(bounds=before.clone())
    want = before.clone()
    for k, q, n in zip(s.keys, s.seq, length):
        ids = s.c.block_table[q, :n // page].long()
        for layer in range(2):
            want[layer, ids] = page_bounds(k[layer], page)
    assert torch.equal(got, want)
    # a step fills the pages between its lengths and touches no others
    step = s.bounds(start=[max(0, n - page - 1) for n in length], bounds=before.clone())
    want = before.clone()
    for k, q, n in zip(s.keys, s.seq, length):
        first = max(0, n - page - 1) // page
        ids = s.c.block_table[q, first:n // page].long()
        for layer in range(2):
            want[layer, ids] = page_bounds(k[layer], page)[first:]
    assert torch.equal(step, want)
    assert dspark.read_device_error(s.c) == 0
    fresh = s.bounds()
    assert fresh.shape == got.shape and torch.equal(torch.where(got == 7.0, 0.0, got), torch.where(fresh == 7.0, 0.0, fresh))


def test_bounds_of_special_keys(cuda):
    """Infinities are bounds like others; a NaN makes its dimension's NaN."""
    s = Case(BF, 64, 2, 1, 1, [128], 32)
    ids = s.c.block_table[0, :4].long()
    s.c.pool[0, 0, ids[1], 0, 5, 7] = math.inf
    s.c.pool[0, 0, ids[1], 0, 6, 7] = -math.inf
    s.c.pool[0, 0, ids[2], 1, 31, 63] = math.nan
    got = s.bounds()
    assert got[0, ids[1], 0, :, 7].tolist() == [-math.inf, math.inf]
    assert torch.isnan(got[0, ids[2], 1, :, 63]).all()
    assert torch.isnan(got[0, ids]).sum() == 2 and torch.isinf(got[0, ids]).sum() == 2


def test_bounds_follow_forks_and_commits(cuda):
    """Shared pages share their bounds; a fork's own page gets bounds when it is full."""
    page, D = 16, 64
    c = dspark.PagedCache(2, 20, page, 2, D, 3, 6, dtype=F32)
    dspark.cache_reserve(c, ints([40]), 0)
    c.pool.normal_()
    bounds = dspark.cache_bounds(c, ints([0]), ints([40]))
    dspark.cache_fork(c, ints([0]), ints([1]), ints([40]))
    dspark.cache_reserve(c, ints([40, 40]), 8)
    own = int(c.block_table[1, 2])
    c.pool[:, :, own, :, 8:] = torch.randn(2, 2, 2, 8, D, device="cuda")
    before = bounds.clone()
    dspark.cache_bounds(c, ints([40, 40]), ints([40, 48]), bounds=bounds)
    assert torch.equal(bounds[:, own], torch.stack([c.pool[:, 0, own].amin(2), c.pool[:, 0, own].amax(2)], dim=2))
    before[:, own] = bounds[:, own]
    assert torch.equal(bounds, before)
    assert dspark.read_device_error(c) == 0


SHAPES = [  # dtype, D, kv, group, T, lengths, page, count, first, last, shared
    (BF, 128, 2, 4, 1, [6400], 64, 16, 1, 2, False),
    (BF, 128, 2, 4, 8, [0, 63, 64, 2000, 1111], 16, 20, 1, 1, False),
    (BF, 64, 3, 1, 3, [900, 100], 8, 33, 0, 0, False),
    (BF, 64, 1, 32, 5, [700], 16, 9, 0, 1, False),
    (BF, 96, 2, 3, 7, [500, 30], 12, 8, 2, 0, True),
    (BF, 128, 1, 8, 61, [1000, 0, 300], 32, 7, 0, 0, True),
    (BF, 128, 2, 8, 64, [650], 32, 5, 1, 0, False),
    (BF, 256, 1, 2, 2, [400], 16, 6, 0, 0, False),
    (BF, 72, 2, 5, 3, [300, 170], 16, 4, 1, 1, False),   # dims of the next larger form
    (BF, 96, 3, 4, 8, [2000, 63, 1111], 16, 20, 1, 1, False),
    (BF, 120, 1, 8, 61, [1000, 0, 300], 32, 7, 0, 0, True),
    (BF, 40, 2, 3, 5, [900, 100], 8, 33, 0, 0, False),
    (BF, 8, 2, 8, 64, [650], 32, 5, 1, 0, False),
    (BF, 136, 2, 5, 3, [300, 170], 16, 4, 1, 1, False),  # FFMA: dim
    (F32, 64, 2, 3, 7, [500, 777], 16, 12, 0, 0, False),
    (F32, 128, 1, 8, 9, [300], 4, 31, 3, 3, True),
    (F32, 40, 1, 32, 3, [70], 1, 10, 0, 0, False),
    (F32, 256, 2, 1, 1, [640], 8, 1, 0, 0, False),
]


@pytest.mark.parametrize("wide", [0, 300, 5000])  # forms for short and long tables
@pytest.mark.parametrize("dtype,D,kv,group,T,length,page,count,first,last,shared", SHAPES)
def test_selects_the_best(cuda, wide, dtype, D, kv, group, T, length, page, count, first, last, shared):
    tokens = [T if b == 0 else (b * 5) % (T + 1) for b in range(len(length))]
    s = Case(dtype, D, kv, group, T, length, page, count=tokens, seq=[len(length) - b for b in range(len(length))],
             seed=D + T, wide=wide)
    bounds = s.bounds()
    out = torch.full((s.B, 1 if shared else T, kv, count), -9, dtype=torch.int32, device="cuda")
    got = dspark.select_pages(s.c, 1, bounds, s.q, ints(length), count, first=first, last=last, shared=shared,
                              token_count=ints(tokens), seq=ints(s.seq), pages=out)
    assert got is out
    s.check(bounds, got, count, first, last, shared)
    for b, t in enumerate(tokens):  # lists behind the last token
        assert (got[b, (1 if t else 0) if shared else t:] == -9).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_long_tables(cuda, dtype):
    """More pages than a thread of the larger form holds."""
    s = Case(dtype, 32, 1, 2, 2, [9001, 2500], 2, seed=4)
    bounds = s.bounds()
    for count in (3, 100, 2500):
        s.check(bounds, dspark.select_pages(s.c, 1, bounds, s.q, ints(s.length), count, last=2), count, 0, 2)


@pytest.mark.parametrize("wide", [0, 300])
@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("kind", ["equal", "zero", "two values", "near"])
def test_scores_on_the_border(cuda, kind, dtype, wide):
    """Equal scores go to the lower page; differences below the error of a
    float32 sum decide."""
    s = Case(dtype, 64, 2, 2, 2, [1600], 16, seed=9, wide=wide)
    bounds = s.bounds()
    ids = s.c.block_table[0, :100].long()
    if kind == "zero":
        bounds[1, ids] = 0
    elif kind == "equal":
        bounds[1, ids] = bounds[1, ids[:1]]
    elif kind == "two values":
        pick = torch.from_numpy(np.random.default_rng(1).integers(0, 2, 100)).cuda()
        bounds[1, ids] = bounds[1, ids[:2]][pick]
    else:  # one small dimension differs, 2^-20 of the scores
        bounds[1, ids] = bounds[1, ids[:1]]
        s.q[..., 63] = 2.0 ** -20
        bounds[1, ids, :, :, 63] = torch.randn(100, 2, 2, device="cuda").to(dtype).sort(dim=-1).values
    for count in (1, 7, 50, 99):
        got = dspark.select_pages(s.c, 1, bounds, s.q, ints([1600]), count)
        s.check(bounds, got, count)


def test_special_scores(cuda):
    """What is not a number counts as infinite; infinite scores are equal."""
    s = Case(BF, 64, 1, 2, 1, [800], 16, seed=3)
    bounds = s.bounds()
    ids = s.c.block_table[0, :50].long()
    bounds[1, ids[40], 0, 1, 3] = math.nan
    bounds[1, ids[30], 0, :, 5] = math.inf
    bounds[1, ids[20], 0, 0, 5] = -math.inf
    s.q[..., 5] = 1.0
    for count in (1, 2, 5):
        s.check(bounds, dspark.select_pages(s.c, 1, bounds, s.q, ints([800]), count), count)


def test_bad_entries(cuda):
    """Sequences and lengths out of range leave their lists alone, and say so;
    others are served."""
    s = Case(BF, 64, 1, 2, 2, [800, 320, 160], 16, seed=5)
    bounds = s.bounds()
    for length, seq, code in (([801 * 16, 320, 160], None, 7), ([-1, 320, 160], None, 7), ([800, 320, 160], [9, 1, 2], 6)):
        out = torch.full((3, 2, 1, 6), -9, dtype=torch.int32, device="cuda")
        dspark.select_pages(s.c, 1, bounds, s.q, ints(length), 6, seq=None if seq is None else ints(seq), pages=out)
        assert (out[0] == -9).all() and (out[1:] >= 0).all()
        assert dspark.read_device_error(s.c) == code
        kept = torch.full_like(bounds, 3.0)
        dspark.cache_bounds(s.c, ints([0, 0, 0]), ints(length), bounds=kept, seq=None if seq is None else ints(seq))
        assert (kept[:, s.c.block_table[0, :50].long()] == 3.0).all() and dspark.read_device_error(s.c) == code
        assert (kept[:, s.c.block_table[1, :20].long()] != 3.0).any()
    s.c.block_table[1, 4] = 10 ** 6  # names no page
    out = dspark.select_pages(s.c, 1, bounds, s.q, ints(s.length), 19)
    assert (out[1, :, 0] == torch.tensor([j for j in range(20) if j != 4], device="cuda")).all()
    assert dspark.read_device_error(s.c) == 7
    dspark.cache_bounds(s.c, ints([0, 0, 0]), ints(s.length), bounds=bounds)
    assert dspark.read_device_error(s.c) == 7


def test_replays_and_streams(cuda):
    """In a graph, with what it reads changed between replays, and on another
    stream."""
    s = Case(BF, 128, 2, 4, 4, [3000, 1500], 32, seed=6)
    length = ints(s.length)
    bounds, pages = s.bounds(), torch.full((2, 4, 2, 11), -1, dtype=torch.int32, device="cuda")
    ws = dspark.SelectWorkspace(s.c, 2, 4)
    start = ints([0, 0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(side):
        dspark.cache_bounds(s.c, start, length, bounds=bounds)
        dspark.select_pages(s.c, 1, bounds, s.q, length, 11, pages=pages, workspace=ws)
        with torch.cuda.graph(graph, stream=side):
            dspark.cache_bounds(s.c, start, length, bounds=bounds)
            dspark.select_pages(s.c, 1, bounds, s.q, length, 11, pages=pages, workspace=ws)
    torch.cuda.current_stream().wait_stream(side)
    for seed in range(3):
        s.q.normal_()
        s.c.pool[:, 0] = torch.where(torch.isnan(s.c.pool[:, 0]), s.c.pool[:, 0], torch.randn_like(s.c.pool[:, 0]))
        s.length = [3000 - 100 * seed, 1500 - 700 * seed]
        length.copy_(ints(s.length))
        graph.replay()
        s.check(bounds, pages, 11)
        again = dspark.select_pages(s.c, 1, bounds, s.q, length, 11, stream=side)
        side.synchronize()
        assert torch.equal(again, pages)


@pytest.mark.parametrize("D,group,T", [(128, 4, 8), (64, 8, 1), (128, 8, 20)])
def test_a_wait_that_runs_out_is_reported(cuda, monkeypatch, D, group, T):
    """DSPARK_TEST_STALL_WAIT=1 makes the warp that issues the products wait for a
    barrier phase that nothing completes, with a short limit: error 2, a clean
    return, and a cache that the next call can use."""
    s = Case(BF, D, 2, group, T, [3000, 0, 700], 16, seed=T)
    bounds, ws = s.bounds(), dspark.SelectWorkspace(s.c, 3, T)
    want = dspark.select_pages(s.c, 1, bounds, s.q, ints(s.length), 9, workspace=ws)
    s.check(bounds, want, 9)
    monkeypatch.setenv("DSPARK_TEST_STALL_WAIT", "1")
    dspark.select_pages(s.c, 1, bounds, s.q, ints(s.length), 9, workspace=ws)
    torch.cuda.synchronize()
    assert dspark.read_device_error(s.c) == 2 and dspark.read_device_error(s.c) == 0
    monkeypatch.delenv("DSPARK_TEST_STALL_WAIT")
    assert torch.equal(dspark.select_pages(s.c, 1, bounds, s.q, ints(s.length), 9, workspace=ws), want)
    assert dspark.read_device_error(s.c) == 0


# rows of more than one tile of products (64), and more items (128 pages of a key
# head) than the GPU has multiprocessors, so that a block goes through several
@pytest.mark.parametrize("D,kv,group,T,B,shared", [(64, 4, 8, 20, 44, False), (128, 4, 5, 17, 30, True), (96, 2, 32, 5, 70, False),
                                                   (128, 8, 8, 61, 15, True), (64, 3, 7, 64, 40, True)])
def test_items_that_follow_one_another(cuda, D, kv, group, T, B, shared):
    rng = np.random.default_rng(D + T)
    length = [int(x) for x in rng.integers(100, 900, B)]
    length[B // 2], length[0] = 0, 1300
    count = [T] + [int(x) for x in rng.integers(0, T + 1, B - 1)]
    s = Case(BF, D, kv, group, T, length, 2, count=count, seed=T)
    assert sum(-(-(n // 2) // 128) for n, t in zip(length, count) if t and n // 2 > 9) * kv > 160 and T * group > 64
    bounds = s.bounds()
    got = dspark.select_pages(s.c, 1, bounds, s.q, ints(length), 9, first=1, shared=shared, token_count=ints(count))
    s.check(bounds, got, 9, 1, 0, shared)
    for _ in range(5):
        again = dspark.select_pages(s.c, 1, bounds, s.q, ints(length), 9, first=1, shared=shared, token_count=ints(count))
        assert torch.equal(got, again)


@pytest.mark.parametrize("D,group,T", [(128, 4, 8), (64, 8, 20)])
def test_a_warp_that_gives_up_alone(cuda, monkeypatch, D, group, T):
    """DSPARK_TEST_STALL_WAIT=3: one of the four warps that load queries has given
    up, the other three have not.  Their waits for it run out: error 2, a clean
    return, and a cache that the next call can use."""
    s = Case(BF, D, 2, group, T, [3000, 0, 700], 16, seed=T)
    bounds, ws = s.bounds(), dspark.SelectWorkspace(s.c, 3, T)
    want = dspark.select_pages(s.c, 1, bounds, s.q, ints(s.length), 9, workspace=ws)
    monkeypatch.setenv("DSPARK_TEST_STALL_WAIT", "3")
    dspark.select_pages(s.c, 1, bounds, s.q, ints(s.length), 9, workspace=ws)
    torch.cuda.synchronize()
    assert dspark.read_device_error(s.c) == 2 and dspark.read_device_error(s.c) == 0
    monkeypatch.delenv("DSPARK_TEST_STALL_WAIT")
    assert torch.equal(dspark.select_pages(s.c, 1, bounds, s.q, ints(s.length), 9, workspace=ws), want)
    assert dspark.read_device_error(s.c) == 0


# powers of two that queries and bounds are multiplied by: scores that float32 rounds by
# a fixed step, cannot hold at all, or can though one of the two is below its normal numbers
@pytest.mark.parametrize("forms", ["few lists", "many lists"])
@pytest.mark.parametrize("powers", [(-70, -75), (-65, -66), (-60, -64), (-45, -50), (-40, -40), (-30, -32), (-140, 0), (0, -140),
                                    (-140, 55), (60, -140), (-140, -20)])
@pytest.mark.parametrize("dtype", [BF, F32])
def test_small_scores(cuda, dtype, powers, forms):
    """The choice is that of exact scores whatever their size."""
    few = forms == "few lists"
    s = Case(dtype, 64, 2 if few else 4, 2, 2 if few else 4, [1600, 900] if few else [900] * 40, 16, seed=8)
    length = ints(s.length)
    bounds = s.bounds()
    bounds = torch.where(torch.isnan(bounds), 0.0, bounds)
    for_q, for_bounds = (max(p, -131) if dtype is BF else p for p in powers)  # its least number is 2^-133
    s.q = (s.q.double() * 2.0 ** for_q).to(dtype)
    bounds = (bounds.double() * 2.0 ** for_bounds).to(dtype)
    assert (s.q != 0).any() and (bounds != 0).any()
    for count in (1, 7, 50):
        s.check(bounds, dspark.select_pages(s.c, 1, bounds, s.q, length, count), count)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scores_that_are_zero_are_equal(cuda, dtype):
    """Zero queries or bounds of either sign: the lowest pages."""
    s = Case(dtype, 64, 1, 2, 1, [800], 16, seed=8)
    bounds = s.bounds()
    ids = s.c.block_table[0, :50].long()
    q = s.q
    for zero in (0.0, -0.0):
        s.check(bounds, dspark.select_pages(s.c, 1, bounds, q * zero, ints([800]), 7), 7, q=q * 0.0)
        some = bounds.clone()
        some[1, ids] = zero
        some[1, ids[::3]] = 0.0
        s.check(some, dspark.select_pages(s.c, 1, some, q, ints([800]), 7), 7)


# (dims, tokens) of two threads' calls: forms of one kernel with different shared memory
@pytest.mark.parametrize("dtype,sizes", [(BF, [(128, 16), (128, 1)]), (BF, [(64, 16), (64, 1)]), (BF, [(256, 3), (136, 3)]),
                                         (F32, [(256, 2), (40, 2)])])
def test_calls_from_two_threads(cuda, dtype, sizes):
    """Each with a cache, a workspace and a stream of its own, all at once."""
    some, errors = [], []
    for D, T in sizes:
        s = Case(dtype, D, 2, 4, T, [800], 16, seed=D)
        bounds, ws = s.bounds(), dspark.SelectWorkspace(s.c, 1, T)
        want = dspark.select_pages(s.c, 1, bounds, s.q, ints([800]), 9, workspace=ws)
        s.check(bounds, want, 9)
        some.append((s, bounds, ws, want, ints([800]), torch.empty_like(want), torch.cuda.Stream()))
    torch.cuda.synchronize()
    start = threading.Barrier(len(some))

    def work(s, bounds, ws, want, length, out, stream):
        try:
            start.wait()
            for _ in range(5000):
                dspark.select_pages(s.c, 1, bounds, s.q, length, 9, pages=out, workspace=ws, stream=stream)
        except Exception as e:
            errors.append(e)
    threads = [threading.Thread(target=work, args=x) for x in some]
    every, _ = sys.getswitchinterval(), sys.setswitchinterval(1e-5)
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    sys.setswitchinterval(every)
    torch.cuda.synchronize()
    assert not errors, errors
    for s, _, _, want, _, out, _ in some:
        assert torch.equal(out, want) and dspark.read_device_error(s.c) == 0
