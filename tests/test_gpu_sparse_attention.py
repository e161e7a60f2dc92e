"""Attention over selected pages of the cache, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.cache_ref import attend_bounds, place, tree_sees
from tests.test_gpu_tree_attention import Case, ints
from tests.test_gpu_tree_units import attend_all

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


class Sparse(Case):
    """Random lists of a sequence's full pages for each token and key head (or
    one for all its tokens): most of them shared by the tokens, some listed
    twice, in any order, with entries of -1 among them."""

    def __init__(self, dtype, D, kv, group, T, length, page, mask="causal", lists=None, width=6, agree=0.7, **more):
        super().__init__(dtype, D, kv, group, T, length, page, mask, **more)
        self.page, self.kv_heads = page, kv
        self.lists = T if lists is None else lists
        rng = np.random.default_rng(T + D + len(length))
        pages = np.full((self.B, self.lists, kv, width), -1, dtype=np.int32)
        for b, n in enumerate(length):
            F = n // page
            for h in range(kv):
                pool = rng.permutation(F)[:width]
                for i in range(self.lists):
                    some = [int(p) for p in pool if rng.random() < agree]
                    some += [int(p) for p in rng.permutation(F)[:width - len(some)] if rng.random() < 0.3]
                    if some and len(some) < width:
                        some.append(some[0])
                    rng.shuffle(some)
                    at = sorted(rng.permutation(width)[:len(some)])
                    pages[b, i, h, at] = some
        self.pages = torch.from_numpy(pages).cuda()

    def run(self, **over):
        a = dict(mask=self.mask, token_count=ints(self.count), seq=ints(self.seq), with_lse=True)
        pages = over.pop("pages", self.pages)
        a.update(over)
        return dspark.sparse_attention(self.c, self.layer, self.q, ints(self.length), pages, **a)

    def sees(self, b):
        """[kv, 1, tokens, keys] which keys each token sees for each key head."""
        n, t = self.length[b], self.count[b]
        F = n // self.page
        sees = tree_sees(n, t, self.words[b], 0, self.position[b])[None].repeat(self.kv_heads, 1, 1)
        pages = self.pages[b].cpu().long().transpose(0, 1)[:, :t]  # [kv, lists, width]
        named = torch.zeros(self.kv_heads, pages.shape[1], F + 1, dtype=torch.bool)
        named.scatter_(2, torch.where((pages < 0) | (pages >= F), F, pages), True)
        sees[:, :, :F * self.page] = named[:, :, :F].repeat_interleave(self.page, dim=2)
        return sees[:, None].cuda()

    def check(self, out, lse, scale=None, error=0):
        scale = scale or 1.0 / math.sqrt(self.D)
        for b in range(self.B):
            t = self.count[b]
            if not t:
                continue
            sees = self.sees(b)
            k, v = (x.nan_to_num(0.0, 0.0, 0.0) for x in (self.k[b], self.v[b]))
            ro, rl, size, reach = attend_all(k.cuda(), v.cuda(), self.q[b, :t], sees, scale)
            bo, bl = attend_bounds(size, reach, ro, rl, sees.shape[-1], self.D, self.c.dtype == BF)
            none = torch.isinf(rl)
            o, l = out[b, :t].double(), lse[b, :t].double()
            assert torch.equal(torch.isinf(l), none), b
            assert (o[none] == 0).all(), b
            assert ((o - ro).abs() <= bo).all(), (b, ((o - ro).abs() / bo).max())
            assert ((l - rl).abs()[~none] <= bl[~none]).all(), b
        assert dspark.read_device_error(self.c) == error


SHAPES = [  # dtype, D, kv, group, T, lengths, page, mask, lists, width
    (BF, 128, 2, 4, 1, [1000], 64, "causal", None, 5),
    (BF, 128, 2, 4, 8, [0, 63, 64, 700, 2000], 64, "causal", None, 6),
    (BF, 128, 1, 8, 61, [300, 0, 640], 32, "tree", 1, 7),
    (BF, 128, 1, 8, 61, [300, 33], 32, "tree", None, 3),
    (BF, 128, 3, 1, 1, [0, 1, 127, 128, 129, 255], 8, "causal", None, 9),
    (BF, 64, 2, 5, 7, [30, 0, 1000], 16, "full", None, 20),
    (BF, 64, 4, 8, 1, [700, 3], 128, "causal", None, 2),
    (BF, 64, 1, 32, 9, [200, 129], 64, "holes", None, 2),
    (BF, 128, 2, 7, 19, [1111, 0, 90], 256, "holes", None, 3),
    (BF, 128, 2, 3, 64, [500, 100], 8, "tree", None, 11),
    (BF, 64, 1, 1, 64, [1200], 512, "holes", 1, 2),
    (BF, 128, 1, 1, 2, [3000], 16, "causal", None, 40),
    (BF, 96, 2, 3, 6, [177, 0], 16, "tree", None, 4),        # dims of the next larger form
    (BF, 96, 1, 8, 61, [300, 0, 640], 32, "tree", 1, 7),
    (BF, 96, 2, 5, 7, [30, 0, 1000], 16, "full", None, 20),
    (BF, 80, 3, 1, 1, [0, 1, 127, 128, 129, 255], 8, "causal", None, 9),
    (BF, 112, 2, 7, 19, [1111, 0, 90], 256, "holes", None, 3),
    (BF, 48, 1, 32, 9, [200, 129], 64, "holes", None, 2),
    (BF, 32, 4, 8, 1, [700, 3], 128, "causal", None, 2),
    (BF, 16, 2, 3, 64, [500, 100], 8, "tree", None, 11),
    (BF, 72, 2, 3, 6, [177, 0], 16, "tree", None, 4),        # FFMA: dim
    (BF, 128, 1, 4, 5, [50, 130], 12, "tree", None, 4),      # FFMA: page
    (BF, 256, 1, 2, 4, [165], 32, "causal", 1, 3),
    (BF, 8, 1, 2, 3, [10, 200], 16, "tree", None, 5),
    (F32, 64, 2, 3, 7, [0, 777, 64], 16, "full", None, 12),
    (F32, 128, 1, 8, 33, [190, 5], 64, "tree", None, 2),
    (F32, 128, 2, 1, 1, [0, 63, 64, 65], 7, "causal", None, 4),
    (F32, 256, 1, 2, 6, [100], 16, "holes", None, 3),
    (F32, 40, 1, 32, 3, [70], 1, "causal", None, 20),
]


@pytest.mark.parametrize("dtype,D,kv,group,T,length,page,mask,lists,width", SHAPES)
def test_matches_64_bits(cuda, dtype, D, kv, group, T, length, page, mask, lists, width):
    s = Sparse(dtype, D, kv, group, T, length, page, mask, lists=lists, width=width, seed=T + D)
    got = s.run()
    s.check(*got)
    again = s.run()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pages_that_no_list_names_are_not_read(cuda, dtype):
    """NaN in them, and in what lies behind the sequences."""
    s = Sparse(dtype, 64, 2, 4, 5, [400, 333], 16, "tree", width=7, seed=5)
    got = s.run()
    for b in range(2):
        for p in range(s.length[b] // 16):
            for h in range(2):
                if not (s.pages[b, :, h] == p).any():
                    s.c.pool[:, :, s.c.block_table[b, p].long(), h] = math.nan
    again = s.run()
    assert torch.equal(got[0], again[0]) and torch.equal(got[1], again[1])
    s.check(*again)


@pytest.mark.parametrize("dtype,D,group,T,page", [(BF, 96, 2, 6, 32), (BF, 48, 8, 40, 16), (BF, 128, 2, 6, 32), (BF, 128, 8, 9, 16), (BF, 64, 4, 50, 64),
                                                  (F32, 64, 2, 6, 16), (BF, 96, 2, 6, 16)])
def test_special_values_reach_who_lists_them(cuda, dtype, D, group, T, page):
    """NaN and infinities in pages that some tokens list reach those and no
    others; the others' results are the same bits as without them."""
    s = Sparse(dtype, D, 1, group, T, [20 * page, 9 * page + 3], page, "causal", width=8, agree=0.5, seed=2)
    clean = s.run()
    hit = [[set() for _ in range(T)] for _ in range(2)]
    for b in range(2):
        F = s.length[b] // page
        for p in range(0, F, 3):
            who = [i for i in range(T) if (s.pages[b, i, 0] == p).any()]
            if not who or len(who) == T:
                continue
            at = s.c.block_table[b, p].long()
            s.c.pool[s.layer, 1, at, 0, p % page, 3] = math.nan if p % 2 else math.inf
            for i in who:
                hit[b][i].add(p)
    assert any(x for y in hit for x in y)
    out, lse = s.run()
    assert torch.equal(lse, clean[1])
    keep = [d for d in range(D) if d != 3]
    assert torch.equal(out[..., keep], clean[0][..., keep])
    for b in range(2):
        for i in range(T):
            x = out[b, i, :, 3]
            if not hit[b][i]:
                assert torch.equal(x, clean[0][b, i, :, 3])
            else:
                assert (~torch.isfinite(x)).all()
    assert dspark.read_device_error(s.c) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padding_and_order(cuda, dtype):
    """Fewer tokens than T, none at all, sequences in another order: rows
    behind the last token stay as they were, whatever their lists hold."""
    s = Sparse(dtype, 64, 2, 4, 8, [160, 37, 300, 0], 16, "causal", count=[8, 0, 3, 1], seq=[5, 0, 3, 1])
    for b, n in enumerate(s.count):
        s.pages[b, n:] = 10 ** 6
    out = torch.full((4, 8, 8, 64), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((4, 8, 8), 6.0, device="cuda")
    got = s.run(out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    s.check(out, lse)
    for b, n in enumerate(s.count):
        assert (out[b, n:] == 5).all() and (lse[b, n:] == 6).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_all_pages_are_the_whole_context(cuda, dtype):
    """Lists of all full pages give what tree_attention gives."""
    s = Sparse(dtype, 128, 2, 4, 8, [500, 129, 0], 32, "tree", width=15)
    s.pages = torch.arange(15, dtype=torch.int32, device="cuda").expand(3, 1, 2, 15).contiguous()
    s.pages = torch.where(s.pages < ints([n // 32 for n in s.length])[:, None, None, None], s.pages, -1)
    s.lists = 1
    got = s.run()
    s.check(*got)
    want = dspark.tree_attention(s.c, s.layer, s.q, ints(s.length), mask=s.mask, with_lse=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_scales_masks_and_empty_lists(cuda, dtype):
    s = Sparse(dtype, 64, 1, 2, 5, [96, 100], 32, "holes", width=3, agree=0.0)
    s.check(*s.run())
    s.check(*s.run(scale=0.3), scale=0.3)
    s.check(*s.run(scale=-0.05), scale=-0.05)
    s.pages.fill_(-1)  # nothing but the tail; a token that sees none of that has zeros
    s.check(*s.run())
    s.words = [[(2 << t) - 1 for t in range(5)]] * 2
    s.check(*s.run(mask=None))


@pytest.mark.parametrize("dtype,page", [(BF, 16), (F32, 16)])
def test_long_lists_of_a_long_context(cuda, dtype, page):
    """More pages than one range of the lists' kernel holds, one sequence over many
    blocks and many sequences a block."""
    s = Sparse(dtype, 64, 2, 2, 3, [20 * 1024 + 5, 17 * 1024, 40], page, "causal", width=300)
    s.check(*s.run())
    rng = np.random.default_rng(0)
    s = Sparse(dtype, 64, 2, 2, 2, [int(x) for x in rng.integers(0, 300, 300)], page, "causal", width=6)
    s.check(*s.run())


# head_dim, key heads, heads of each, tokens: 8, 48 and 192 rows
FORMS = [(128, 8, 1, 8), (64, 8, 1, 8), (128, 8, 8, 6), (64, 8, 8, 6), (128, 8, 3, 64), (64, 8, 3, 64),
         (96, 8, 1, 8), (48, 8, 8, 6), (112, 8, 3, 64)]


@pytest.mark.parametrize("D,kv,group,T", FORMS)
@pytest.mark.parametrize("page", [8, 64])
def test_units_that_follow_one_another(cuda, D, kv, group, T, page):
    """Several units of one to several tiles in each block, with NaN behind the
    sequences and infinities in pages that not all tokens see."""
    rng = np.random.default_rng(D + T)
    length = [int(x) for x in rng.integers(1, 900, 88)]
    count = [int(x) for x in rng.integers(1, T + 1, 88)]
    s = Sparse(BF, D, kv, group, T, length, page, "causal", width=512 // page, agree=0.8, count=count, seed=D)
    out, lse = torch.zeros_like(s.q), torch.zeros(88, T, kv * group, device="cuda")
    s.run(out=out, lse=lse)
    s.check(out, lse)
    again, again_lse = torch.zeros_like(out), torch.zeros_like(lse)
    for _ in range(5):
        s.run(out=again, lse=again_lse)
        assert torch.equal(out, again) and torch.equal(lse, again_lse)


@pytest.mark.parametrize("dtype", [BF, F32])
def test_bad_entries(cuda, dtype):
    s = Sparse(dtype, 64, 1, 2, 4, [130, 64, 260], 16, width=5)
    good = s.run()
    for bad, code in ((dict(seq=ints([0, 9, 2])), 6), (dict(seq=ints([0, -1, 2])), 6)):
        out = torch.full_like(s.q, 3.0)
        s.run(out=out, **bad)
        assert dspark.read_device_error(s.c) == code
        assert (out[1] == 3).all() and torch.equal(out[0], good[0][0]) and torch.equal(out[2], good[0][2])
    for n in (-1, 1000, 2147483647):
        out, kept = torch.full_like(s.q, 3.0), s.length
        s.length = [130, n, 260]
        s.run(out=out)
        s.length = kept
        assert dspark.read_device_error(s.c) == 7 and (out[1] == 3).all() and torch.equal(out[0], good[0][0])
    for page in (8, 9, 2147483647):  # behind the full pages: passed over
        pages = s.pages.clone()
        pages[0, :, :, :][pages[0] == -1] = page
        assert (pages != s.pages).any()
        again = s.run(pages=pages)
        assert dspark.read_device_error(s.c) == 7
        assert torch.equal(again[0], good[0]) and torch.equal(again[1], good[1])
    s.c.block_table[1, :4] = 1 << 30
    out = s.run()[0]
    assert dspark.read_device_error(s.c) == 7 and torch.equal(out[0], good[0][0])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("lists", [1, 3])
def test_entries_of_a_sequence_without_full_pages(cuda, dtype, lists):
    c = dspark.PagedCache(1, 4, 16, 2, 64, 1, 4, dtype=dtype)
    c.pool.normal_()
    n = torch.tensor([9], dtype=torch.int32, device="cuda")
    dspark.cache_reserve(c, n, 3)
    q = torch.randn(1, 3, 4, 64, device="cuda").to(dtype)
    none = torch.full((1, lists, 2, 5), -1, dtype=torch.int32, device="cuda")
    want = dspark.sparse_attention(c, 0, q, n, none)[0]
    assert dspark.read_device_error(c) == 0
    none[0, lists - 1, 1, 2] = 0
    assert torch.equal(dspark.sparse_attention(c, 0, q, n, none)[0], want)
    assert dspark.read_device_error(c) == 7


@pytest.mark.parametrize("dtype", [BF, F32])
def test_graph_replay_and_streams(cuda, dtype):
    """A captured call reads lengths, lists and masks anew, and two graphs with
    workspaces of their own replay in any order; another stream; a workspace that a
    larger call shares."""
    s = Sparse(dtype, 128, 2, 2, 8, [200, 140], 16, "tree")
    length, count = ints(s.length), ints(s.count)
    out = [torch.zeros_like(s.q) for _ in range(2)]
    lse = [torch.zeros(2, 8, 4, device="cuda") for _ in range(2)]
    ws = [dspark.SparseWorkspace(s.c, 3, 16, 4, 30) for _ in range(2)]

    def call(i):
        dspark.sparse_attention(s.c, s.layer, s.q, length, s.pages, mask=s.mask, token_count=count, out=out[i],
                                lse=lse[i], workspace=ws[i])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call(0)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            call(i)
    for turn in range(3):
        for g in graphs[::-1]:
            g.replay()
        torch.cuda.synchronize()
        for i in range(2):
            s.check(out[i], lse[i])
        s.pages.copy_(s.pages.roll(1, dims=1))
        count.copy_(ints([8 - turn, 3 + turn]))
        s.count = [8 - turn, 3 + turn]
        for b in range(2):
            n = s.length[b] + s.count[b]
            ids, slots = place(s.c, b, n)
            s.k[b] = s.c.pool[s.layer, 0][ids.cuda(), :, slots.cuda()].transpose(0, 1).cpu()
            s.v[b] = s.c.pool[s.layer, 1][ids.cuda(), :, slots.cuda()].transpose(0, 1).cpu()
    want = s.run()
    torch.cuda.synchronize()
    got, _ = dspark.sparse_attention(s.c, s.layer, s.q, length, s.pages, mask=s.mask, token_count=count, stream=stream)
    stream.synchronize()
    for b, n in enumerate(s.count):
        assert torch.equal(got[b, :n], want[0][b, :n])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_step_as_it_is_used(cuda, dtype):
    """Bounds behind what is committed, pages selected by them, and the attention
    over these: the result is that over the best pages."""
    s = Sparse(dtype, 64, 2, 4, 6, [1000, 333, 0], 16, "causal", width=9)
    length = ints(s.length)
    bounds = dspark.cache_bounds(s.c, ints([0, 0, 0]), length)
    for shared in (False, True):
        s.pages = dspark.select_pages(s.c, s.layer, bounds, s.q, length, 9, first=1, last=1, shared=shared)
        s.lists = 1 if shared else 6
        for b in (0, 1):  # the first and last full pages are there
            got = s.pages[b, 0, 0].tolist()
            assert got[0] == 0 and got[-1] == s.length[b] // 16 - 1 and got == sorted(set(got))
        s.check(*s.run())


@pytest.mark.parametrize("D,group,T", [(128, 4, 8), (64, 8, 6), (64, 5, 40)])
def test_a_wait_that_runs_out_is_reported(cuda, monkeypatch, D, group, T):
    s = Sparse(BF, D, 4, group, T, [700, 130, 0, 1000], 16, "causal", seed=T, width=12)
    a = dict(out=torch.zeros_like(s.q), lse=torch.zeros(4, T, 4 * group, device="cuda"),
             workspace=dspark.SparseWorkspace(s.c, 4, T, 4 * group, 12))
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


@pytest.mark.parametrize("D,kv,group,T", [(64, 8, 4, 1), (128, 8, 2, 3), (96, 4, 8, 4)])
def test_a_stream_that_is_late(cuda, monkeypatch, D, kv, group, T):
    """Units of one tile leave the second stream without work.  With
    DSPARK_TEST_STALL_WAIT=2 its warps come to each unit's end long after the
    others: the same results, and no wait runs out."""
    rng = np.random.default_rng(D)
    length = [int(n) for n in rng.integers(0, 120, 240)]
    for b in range(0, 240, 9):  # and some units of two to four tiles
        length[b] = int(rng.integers(130, 400))
    s = Sparse(BF, D, kv, group, T, length, 16, "causal", width=24, seed=D)
    a = dict(out=torch.zeros_like(s.q), lse=torch.zeros(240, T, kv * group, device="cuda"),
             workspace=dspark.SparseWorkspace(s.c, 240, T, kv * group, 24))
    s.run(**a)
    s.check(a["out"], a["lse"])
    want = [a["out"].clone(), a["lse"].clone()]
    monkeypatch.setenv("DSPARK_TEST_STALL_WAIT", "2")
    for _ in range(3):
        a["out"].zero_()
        s.run(**a)
        torch.cuda.synchronize()
        assert dspark.read_device_error(s.c) == 0
        assert torch.equal(a["out"], want[0]) and torch.equal(a["lse"], want[1])
