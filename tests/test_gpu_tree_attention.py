"""Attention of drafted tokens over the paged cache, against 64 bits."""
import math

import numpy as np
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.cache_ref import (as_int64, attend, attend_bounds, place, rotate, tree_sees, tree_words)

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Case:
    """A cache with random contents whose sequences hold what a call needs,
    and NaN everywhere that the call must not look at."""

    def __init__(self, dtype, D, kv, group, T, length, page, mask="causal", count=None, window=0,
                 seq=None, seed=0, layers=2, poison=True):
        self.rng = np.random.default_rng(seed)
        g = torch.Generator(device="cuda").manual_seed(seed)
        self.B, self.T, self.heads, self.D, self.kv = len(length), T, kv * group, D, kv
        self.length, self.window = length, window
        self.count = count or [T] * self.B
        self.seq = seq or list(range(self.B))
        pages = sum(-(-(n + T) // page) + 1 for n in length)
        widest = max(-(-(n + T) // page) for n in length) + 2
        self.c = c = dspark.PagedCache(layers, pages + 3, page, kv, D, max(self.seq) + 2, widest, dtype=dtype)
        # a stack in random order: pages lie scattered
        c.free_list.copy_(torch.randperm(pages + 3, generator=g, device="cuda").int())
        dspark.cache_reserve(c, ints(length), T, seq=ints(self.seq))
        if poison:
            c.pool.fill_(float("nan"))
        layer = layers - 1
        self.layer = layer
        self.q = torch.randn(self.B, T, self.heads, D, generator=g, device="cuda").to(dtype)
        self.k, self.v = [], []
        for b, s in enumerate(self.seq):
            n = length[b] + self.count[b]
            k = torch.randn(kv, n, D, generator=g, device="cuda").to(dtype)
            v = torch.randn(kv, n, D, generator=g, device="cuda").to(dtype)
            ids, slots = place(c, s, n)
            for plane, x in ((0, k), (1, v)):
                c.pool[layer, plane][ids.cuda(), :, slots.cuda()] = x.transpose(0, 1)
            self.k.append(k.cpu())
            self.v.append(v.cpu())
        words = [tree_words(mask, T, self.rng) for _ in range(self.B)]
        self.words = [w for w, _ in words]
        self.position = [[n + d for d in depth] for n, (_, depth) in zip(length, words)]
        self.mask = as_int64(self.words).cuda()

    def run(self, **over):
        a = dict(mask=self.mask, position=ints(self.position), window=self.window,
                 token_count=ints(self.count), seq=ints(self.seq), with_lse=True)
        a.update(over)
        return dspark.tree_attention(self.c, self.layer, self.q, ints(self.length), **a)

    def check(self, out, lse, scale=None):
        scale = scale or 1.0 / math.sqrt(self.D)
        out, lse = out.double().cpu(), lse.double().cpu()
        for b in range(self.B):
            t = self.count[b]
            if not t:
                continue
            sees = tree_sees(self.length[b], t, self.words[b], self.window, self.position[b])
            ro, rl, size, reach = attend(self.k[b], self.v[b], self.q[b, :t].cpu(), sees, scale)
            bo, bl = attend_bounds(size, reach, ro, rl, sees.shape[1], self.D, self.c.dtype == torch.bfloat16)
            assert torch.equal(torch.isinf(lse[b, :t]), torch.isinf(rl)), b
            none = torch.isinf(rl)
            assert (out[b, :t][none] == 0).all()
            assert ((out[b, :t] - ro).abs() <= bo).all(), (b, ((out[b, :t] - ro).abs() / bo).max())
            dl = (lse[b, :t] - rl).abs()[~none]
            assert (dl <= bl[~none]).all(), b
        assert dspark.read_device_error(self.c) == 0


BF, F32 = torch.bfloat16, torch.float32
SHAPES = [  # dtype, D, kv, group, T, lengths, page, mask
    (BF, 128, 2, 4, 8, [0, 1, 100, 128, 500], 64, "causal"),
    (BF, 128, 1, 8, 61, [0, 300, 67, 121], 32, "tree"),
    (BF, 128, 1, 3, 64, [127, 64], 16, "tree"),
    (BF, 128, 3, 1, 1, [0, 1, 127, 128, 129, 255], 8, "causal"),
    (BF, 64, 2, 5, 7, [30, 0, 1000], 16, "full"),
    (BF, 64, 4, 8, 1, [700, 3], 128, "causal"),
    (BF, 64, 1, 32, 9, [200, 129], 64, "holes"),
    (BF, 128, 2, 7, 19, [511, 0, 90], 256, "holes"),
    (BF, 128, 1, 1, 2, [3000], 16, "causal"),
    (BF, 96, 2, 3, 6, [77, 0], 16, "tree"),        # FFMA: dim
    (BF, 128, 1, 4, 5, [50, 130], 12, "tree"),     # FFMA: page
    (BF, 256, 1, 2, 4, [65], 32, "causal"),
    (BF, 8, 1, 2, 3, [10, 200], 16, "tree"),
    (F32, 64, 2, 3, 7, [0, 777, 64], 16, "full"),
    (F32, 128, 1, 8, 33, [190, 5], 64, "tree"),
    (F32, 128, 2, 1, 1, [0, 63, 64, 65], 7, "causal"),
    (F32, 256, 1, 2, 6, [100], 16, "holes"),
    (F32, 40, 1, 32, 3, [70], 1, "causal"),
]


@pytest.mark.parametrize("dtype,D,kv,group,T,length,page,mask", SHAPES)
def test_matches_64_bits(cuda, dtype, D, kv, group, T, length, page, mask):
    s = Case(dtype, D, kv, group, T, length, page, mask, seed=T + D)
    s.check(*s.run())


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("window", [1, 5, 64, 100, 129, 10000])
def test_windows(cuda, dtype, window):
    s = Case(dtype, 128, 2, 2, 9, [0, 50, 400, 128], 16, "tree", window=window, seed=window)
    s.check(*s.run())
    if window == 100:  # a position below the length counts as the length
        s.position = [[0] * 9] * 4
        s.check(*s.run())
        s.position = [[n + t for t in range(9)] for n in s.length]
        s.check(*s.run(position=None))


@pytest.mark.parametrize("dtype", [BF, F32])
def test_padding_and_order(cuda, dtype):
    """Fewer tokens than T, none at all, sequences in another order: rows
    behind the last token stay as they were."""
    s = Case(dtype, 64, 2, 4, 8, [60, 7, 300, 0], 16, "causal", count=[8, 0, 3, 1], seq=[5, 0, 3, 1])
    out = torch.full((4, 8, 8, 64), 5.0, dtype=dtype, device="cuda")
    lse = torch.full((4, 8, 8), 6.0, device="cuda")
    got = s.run(out=out, lse=lse)
    assert got[0] is out and got[1] is lse
    s.check(out, lse)
    for b, n in enumerate(s.count):
        assert (out[b, n:] == 5).all() and (lse[b, n:] == 6).all()


@pytest.mark.parametrize("dtype", [BF, F32])
def test_default_mask_scale_and_shared_tree(cuda, dtype):
    s = Case(dtype, 128, 1, 2, 64, [100, 3], 32, "causal")
    s.check(*s.run(mask=None))
    s.check(*s.run(mask=s.mask[0].contiguous()))
    s.check(*s.run(scale=0.3), scale=0.3)
    s.check(*s.run(scale=-0.05), scale=-0.05)
    a, none = s.run(with_lse=False)
    assert none is None and torch.equal(a, s.run()[0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_special_values_stay_where_they_are_seen(cuda, dtype):
    """A drafted token whose keys and values are NaN or infinite reaches the
    tokens that see it and no other."""
    s = Case(dtype, 128, 1, 2, 6, [130, 40, 0], 16, "tree", seed=3)
    clean = s.run()[0].float()
    for bad in (float("nan"), float("inf"), -float("inf")):
        for b in range(3):
            j = 3
            ids, slots = place(s.c, b, s.length[b] + 6)
            s.c.pool[s.layer, 1, ids[s.length[b] + j], 0, slots[s.length[b] + j], 7] = bad
            s.c.pool[s.layer, 1, ids[s.length[b] + j], 0, slots[s.length[b] + j], 100] = bad
        out = s.run()[0].float()
        for b in range(3):
            for t in range(6):
                if (s.words[b][t] >> 3) & 1:
                    want = out[b, t, :, 7]
                    assert (torch.isnan(want) if math.isnan(bad) else want == bad).all()
                    rest = [d for d in range(128) if d not in (7, 100)]
                    assert torch.isfinite(out[b, t][:, rest]).all()
                else:
                    assert torch.equal(out[b, t], clean[b, t])
    for b in range(3):
        ids, slots = place(s.c, b, s.length[b] + 6)
        s.c.pool[s.layer, 0, ids[s.length[b] + 3], 0, slots[s.length[b] + 3]] = float("nan")
        s.c.pool[s.layer, 1, ids[s.length[b] + 3], 0, slots[s.length[b] + 3]] = 0.0
    out = s.run()[0].float()
    for b in range(3):
        for t in range(6):
            if (s.words[b][t] >> 3) & 1:
                assert torch.isnan(out[b, t]).all()
            else:
                assert torch.equal(out[b, t], clean[b, t])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_infinities_behind_a_window(cuda, dtype):
    """Committed tokens that some rows see and others do not."""
    s = Case(dtype, 64, 1, 1, 4, [200], 16, "causal", window=40, seed=9)
    clean = s.run()[0].float()
    # position 200 + t sees tokens from 161 + t on: token 162 by t = 0, 1
    ids, slots = place(s.c, 0, 204)
    s.c.pool[s.layer, 1, ids[162], 0, slots[162], 5] = float("inf")
    s.c.pool[s.layer, 1, ids[20], 0, slots[20]] = float("nan")
    out = s.run()[0].float()
    assert (out[0, :2, 0, 5] == float("inf")).all() and torch.equal(out[0, 2:], clean[0, 2:])
    keep = [d for d in range(64) if d != 5]
    assert torch.equal(out[0, :2][..., keep], clean[0, :2][..., keep])


@pytest.mark.parametrize("dtype", [BF, F32])
@pytest.mark.parametrize("size", [30.0, 3000.0])
def test_large_scores(cuda, dtype, size):
    """Scores that grow along the keys and far past float's exponent range
    of exp: the running maximum carries them."""
    s = Case(dtype, 64, 1, 2, 3, [700], 64, "causal", seed=1)
    ramp = torch.linspace(0.1, 1.0, 703)[None, :, None] * size
    s.k = [(s.k[0].float() * ramp).to(dtype)]
    ids, slots = place(s.c, 0, 703)
    s.c.pool[s.layer, 0][ids.cuda(), :, slots.cuda()] = s.k[0].transpose(0, 1).cuda()
    s.check(*s.run())


@pytest.mark.parametrize("dtype,D", [(BF, 128), (F32, 64)])
def test_many_sequences_and_one_long_one(cuda, dtype, D):
    """More units than blocks, and one unit over many blocks: both ends of
    the split, and the same bits on every run."""
    s = Case(dtype, D, 1, 1, 2, [int(x) for x in np.random.default_rng(0).integers(0, 40, 400)], 16)
    s.check(*s.run())
    s = Case(dtype, D, 1, 2, 3, [20000, 1], 64)
    a, b = s.run(), s.run()
    s.check(*a)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_sequences_out_of_range_are_left(cuda, dtype):
    s = Case(dtype, 64, 1, 2, 4, [30, 10, 60], 16, count=[4, 4, 4])
    good = s.run()
    for bad, code in ((dict(seq=ints([0, 9, 2])), 6), (dict(seq=ints([0, -1, 2])), 6)):
        out, lse = torch.full_like(s.q, 3.0), torch.full((3, 4, 2), 3.0, device="cuda")
        s.run(out=out, lse=lse, **bad)
        assert dspark.read_device_error(s.c) == code
        assert (out[1] == 3).all() and (lse[1] == 3).all()
        assert torch.equal(out[0], good[0][0]) and torch.equal(out[2], good[0][2])
    for n in (-1, 1000, 2147483647):
        out = torch.full_like(s.q, 3.0)
        s2 = s.length
        s.length = [30, n, 60]
        s.run(out=out)
        s.length = s2
        assert dspark.read_device_error(s.c) == 7 and (out[1] == 3).all()
        assert torch.equal(out[0], good[0][0])
    s.c.block_table[1, 0] = 1 << 30
    out = s.run()[0]
    assert dspark.read_device_error(s.c) == 7 and torch.equal(out[0], good[0][0])


@pytest.mark.parametrize("dtype", [BF, F32])
def test_graph_replay_follows_the_lengths(cuda, dtype):
    """A captured call reads lengths, counts and masks anew; two graphs with
    workspaces of their own replay in any order."""
    s = Case(dtype, 128, 2, 2, 8, [200, 40], 16, "tree")
    length, count = ints(s.length), ints(s.count)
    out = [torch.zeros_like(s.q) for _ in range(2)]
    lse = [torch.zeros(2, 8, 4, device="cuda") for _ in range(2)]
    ws = [dspark.TreeWorkspace(2, 8, 4, 2, 128) for _ in range(2)]

    def call(i):
        dspark.tree_attention(s.c, s.layer, s.q, length, mask=s.mask, token_count=count,
                              out=out[i], lse=lse[i], workspace=ws[i])
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        call(0)
    torch.cuda.synchronize()
    graphs = [torch.cuda.CUDAGraph() for _ in range(2)]
    for i, g in enumerate(graphs):
        with torch.cuda.graph(g):
            call(i)
    for g in graphs[::-1]:
        g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        s.check(out[i], lse[i])
    # shorter: the drafted keys now lie inside what was committed before
    count.copy_(ints([3, 8]))
    s.count = [3, 8]
    s.k[0], s.v[0] = s.k[0][:, :203], s.v[0][:, :203]
    for g in graphs:
        g.replay()
    torch.cuda.synchronize()
    for i in range(2):
        s.check(out[i], lse[i])


def test_another_stream(cuda):
    s = Case(BF, 128, 1, 2, 4, [100], 16)
    want = s.run()[0]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    length, pos = ints(s.length), ints(s.position)
    torch.cuda.synchronize()
    got, _ = dspark.tree_attention(s.c, s.layer, s.q, length, mask=s.mask, position=pos, stream=stream)
    stream.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("dtype,tree", [(BF, False), (BF, True), (F32, True)])
def test_decoding_steps(cuda, dtype, tree):
    """The chain as it is used: reserve, append, attend, verify, accept, three
    steps long in two layers, a fork between them.  After each step the
    attention is that of the accepted tokens alone, as if nothing had ever
    been drafted."""
    rng = np.random.default_rng(2)
    g = torch.Generator(device="cuda").manual_seed(2)
    layers, kv, group, D, page, T, V = 2, 2, 3, 64, 16, 8, 50
    heads = kv * group
    c = dspark.PagedCache(layers, 60, page, kv, D, 4, 12, dtype=dtype)
    c.pool.fill_(float("nan"))
    cs = torch.randn(200, D, generator=g, device="cuda")
    w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
    seq, B = ints([2, 0]), 2
    length = ints([0, 0])
    past = [[[] for _ in range(layers)] for _ in range(B)]  # accepted (k, v) rows

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)

    for step in range(3):
        words, depth = tree_words("tree" if tree else "causal", T, rng)
        mask = as_int64(words).cuda()
        n = length.tolist()
        position = ints([[x + d for d in depth] for x in n])
        dspark.cache_reserve(c, length, T, seq=seq)
        fresh = []
        for layer in range(layers):
            q, k, v = normal(B, T, heads, D), normal(B, T, kv, D), normal(B, T, kv, D)
            rq = dspark.cache_append(c, layer, q, k, v, length, position=position, cos_sin=cs,
                                     q_weight=w, k_weight=w, seq=seq)
            out, lse = dspark.tree_attention(c, layer, rq, length, mask=mask, seq=seq, with_lse=True)
            rk = rotate(k.cpu(), w.cpu(), 1e-6, cs.cpu(), position.cpu(), False)[0].to(dtype)
            fresh.append((rk, v.cpu()))
            for b in range(B):
                old = past[b][layer]
                K = torch.stack([x for x, _ in old], 1) if old else torch.zeros(kv, 0, D, dtype=dtype)
                Vv = torch.stack([x for _, x in old], 1) if old else torch.zeros(kv, 0, D, dtype=dtype)
                K = torch.cat([K, rk[b].transpose(0, 1)], 1)
                Vv = torch.cat([Vv, v[b].cpu().transpose(0, 1)], 1)
                sees = tree_sees(n[b], T, words, 0, position[b].tolist())
                ro, rl, size, reach = attend(K, Vv, rq[b].cpu(), sees, 1 / math.sqrt(D))
                bo, bl = attend_bounds(size, reach, ro, rl, sees.shape[1], D, dtype == BF)
                # the reference's keys are rounded from 64 bits: a rounding
                # that falls the other way moves a score by 2^-7 |q||k|
                slack = 2 * (2.0 ** -7 if dtype == BF else 2.0 ** -23) * reach
                bo = bo + slack[..., None] * size
                assert ((out[b].double().cpu() - ro).abs() <= bo).all()
                assert ((lse[b].double().cpu() - rl).abs() <= bl + slack).all()
        # a deepest path is drafted and verified against a target
        t = max(range(T), key=lambda i: depth[i])
        path = [i for i in range(T) if (words[t] >> i) & 1]
        K = len(path) - 1
        drafts = ints(rng.integers(0, V, (B, K)).tolist())
        qp = torch.softmax(torch.randn(B, K, V, generator=g, device="cuda"), -1)
        tp = torch.softmax(torch.randn(B, K + 1, V, generator=g, device="cuda"), -1)
        key = torch.arange(B, device="cuda")
        accepted, _ = dspark.verify_standard(qp, tp, drafts, key, key + step)
        length = dspark.cache_accept(c, length, accepted, T, seq=seq,
                                     path=ints([path] * B) if tree else None)
        for b in range(B):
            keep = int(accepted[b]) + 1
            assert int(length[b]) == n[b] + keep
            for layer in range(layers):
                rk, v = fresh[layer]
                past[b][layer] += [(rk[b, i], v[b, i]) for i in path[:keep]]
        if step == 1:  # the second request goes on as a copy of the first
            dspark.cache_fork(c, ints([2]), ints([1]), length[:1].contiguous())
            dspark.cache_release(c, ints([0]))
            seq = ints([2, 1])
            past[1] = [list(x) for x in past[0]]
            length = length[:1].repeat(2).contiguous()
    assert dspark.read_device_error(c) == 0
    dspark.cache_release(c, seq)
    assert int(c.control[1]) == 60
