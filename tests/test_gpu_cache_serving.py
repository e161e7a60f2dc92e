"""The cache calls as a server makes them: whole steps captured in a graph,
several streams, shared workspaces, the largest batches and pools beyond 4 GB."""
import numpy as np
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.cache_ref import PageModel, as_int64, tree_words

pytestmark = pytest.mark.gpu
BF, F32 = torch.bfloat16, torch.float32


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


class Decoder:
    """Steps of a drafted tree over two layers, all state on the device."""

    def __init__(self, dtype, B=3, T=8, kv=2, group=3, D=64, page=16, num_pages=90, max_pages=20,
                 seed=0, ids=None):
        g = torch.Generator(device="cuda").manual_seed(seed)
        rng = np.random.default_rng(seed)
        self.B, self.T, self.layers = B, T, 2
        self.c = dspark.PagedCache(2, num_pages, page, kv, D, B + 1, max_pages, dtype=dtype)
        if ids is not None:
            self.c.free_list.copy_(ids)
        words, depth = tree_words("tree", T, rng)
        self.mask = as_int64(words).cuda()
        self.depth = ints(depth)
        self.seq = ints([b + 1 for b in range(B)][::-1])
        self.length = ints([0] * B)
        self.position = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        self.accepted = ints([0] * B)
        self.path = torch.zeros(B, T, dtype=torch.int32, device="cuda")
        self.cs = torch.randn(400, D, generator=g, device="cuda")
        self.w = 1 + 0.1 * torch.randn(D, generator=g, device="cuda")
        self.qkv = torch.randn(2, B, T, kv * (group + 2), D, generator=g, device="cuda").to(dtype)
        self.q = torch.empty(2, B, T, kv * group, D, dtype=dtype, device="cuda")
        self.out = torch.empty_like(self.q)
        self.lse = torch.empty(2, B, T, kv * group, device="cuda")
        self.kv, self.heads = kv, kv * group
        self.ws = dspark.TreeWorkspace(B, T, kv * group, kv, D)

    def step(self):
        c, h = self.c, self.heads
        dspark.cache_reserve(c, self.length, self.T, seq=self.seq)
        torch.add(self.length[:, None], self.depth[None], out=self.position)
        for x in range(2):
            q, k, v = self.qkv[x].split([h, self.kv, self.kv], dim=2)
            dspark.cache_append(c, x, q, k, v, self.length, position=self.position, cos_sin=self.cs,
                                q_weight=self.w, k_weight=self.w, seq=self.seq, q_out=self.q[x])
            dspark.tree_attention(c, x, self.q[x], self.length, mask=self.mask, seq=self.seq,
                                  position=self.position, window=70, out=self.out[x],
                                  lse=self.lse[x], workspace=self.ws)
        dspark.cache_accept(c, self.length, self.accepted, self.T, path=self.path, seq=self.seq,
                            new_length=self.length)

    def choose(self, n):
        """What the next step accepts, drawn from n."""
        rng = np.random.default_rng(n)
        acc, path = [], []
        for _ in range(self.B):
            a = int(rng.integers(-1, self.T))
            acc.append(a)
            path.append(sorted(rng.permutation(self.T)[:a + 1].tolist()) + [0] * (self.T - 1 - a))
        self.accepted.copy_(ints(acc))
        self.path.copy_(ints(path))
        # other queries, keys and values
        self.qkv.copy_(self.qkv.roll(1, dims=1).roll(1, dims=2))

    def state(self):
        c = self.c
        held = [c.block_table, c.page_count, c.ref_count, c.control[1:3], self.length, self.out, self.lse]
        rows = []
        for s, n in zip(self.seq.tolist(), self.length.tolist()):
            at = torch.arange(n, device="cuda")
            ids = c.block_table[s].long()[at // c.page_size]
            rows.append(c.pool[:, :, ids, :, at % c.page_size].clone())
        return [x.clone() for x in held] + rows


def same(a, b):
    return len(a) == len(b) and all(torch.equal(x, y) for x, y in zip(a, b))


@pytest.mark.parametrize("dtype,T", [(BF, 8), (BF, 1), (F32, 5)])
def test_whole_step_in_one_graph(cuda, dtype, T):
    """One graph, replayed: everything that changes from step to step is on
    the device.  The same bits as calls one by one."""
    eager, other = Decoder(dtype, T=T), Decoder(dtype, T=T)
    want = []
    for n in range(6):
        eager.choose(n)
        eager.step()
        want.append(eager.state())
    other.choose(0)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other.step()
    torch.cuda.synchronize()
    assert same(other.state(), want[0])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        other.step()
    for n in range(1, 6):
        other.choose(n)
        graph.replay()
        torch.cuda.synchronize()
        assert same(other.state(), want[n]), n
    assert dspark.read_device_error(other.c) == 0 and dspark.read_device_error(eager.c) == 0


def test_two_graphs_take_turns_with_one_workspace(cuda):
    """A workspace holds nothing from one call to the next, so graphs that
    replay one after the other may share it, whatever their sizes."""
    big, small = Decoder(BF, B=4, T=8, seed=3), Decoder(F32, B=1, T=3, seed=4)
    n = max(big.ws.nbytes, small.ws.nbytes)
    ws = dspark.TreeWorkspace(4, 8, 6, 2, 64)
    assert ws.nbytes >= n
    ref = [Decoder(BF, B=4, T=8, seed=3), Decoder(F32, B=1, T=3, seed=4)]
    graphs = []
    for d in (big, small):
        d.ws = ws
        d.choose(0)
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(side):
            d.step()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            d.step()
        graphs.append(graph)
    for r in ref:
        r.choose(0)
        r.step()
    for n in (1, 2, 3):
        for d, r, graph in zip((big, small), ref, graphs):
            d.choose(n)
            r.choose(n)
            graph.replay()
            r.step()
    torch.cuda.synchronize()
    for d, r in zip((big, small), ref):
        assert same(d.state(), r.state())


def test_two_caches_on_two_streams(cuda):
    pair = [Decoder(BF, seed=5), Decoder(F32, seed=6)]
    ref = [Decoder(BF, seed=5), Decoder(F32, seed=6)]
    for d in pair + ref:
        d.choose(1)
    for r in ref:
        for _ in range(3):
            r.step()
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in pair]
    for _ in range(3):
        for d, st in zip(pair, streams):
            with torch.cuda.stream(st):
                d.step()
    torch.cuda.synchronize()
    for d, r in zip(pair, ref):
        assert same(d.state(), r.state())


def test_memory_that_a_call_makes_belongs_to_its_stream(cuda):
    """Scratch that a call on another stream has allocated is not handed out
    again before that stream has come by."""
    d = Decoder(BF, B=3, T=8, seed=7)
    d.choose(2)
    d.step()
    dspark.cache_reserve(d.c, d.length, 8, seq=d.seq)
    want, _ = dspark.tree_attention(d.c, 0, d.q[0], d.length, mask=d.mask, seq=d.seq)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    with torch.cuda.stream(side):
        torch.cuda._sleep(20_000_000)  # some 10 ms
    got, _ = dspark.tree_attention(d.c, 0, d.q[0], d.length, mask=d.mask, seq=d.seq, stream=side)
    trash = [torch.full((d.ws.nbytes,), 0, dtype=torch.uint8, device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    assert torch.equal(got, want)
    assert all(int(t.max()) == 0 for t in trash)
    assert dspark.read_device_error(d.c) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_pages_behind_4_gb(cuda, dtype):
    """The same steps on a small pool and on the last pages of a large one:
    the same bits, a fork's copy among them."""
    per = 2 * 2 * 2 * 16 * 64 * (2 if dtype == BF else 4)  # bytes of a page, all planes
    many = (5 << 30) // per
    near = Decoder(dtype, seed=8)
    far = Decoder(dtype, seed=8, num_pages=many,
                  ids=torch.arange(many, dtype=torch.int32, device="cuda"))  # the last on top
    for d in (near, far):
        for n in range(4):
            d.choose(n)
            d.step()
    assert int(far.c.block_table[int(far.seq[0]), 0]) > many - 100
    assert same(far.state()[4:], near.state()[4:])
    for d in (near, far):
        n = int(d.length.max())
        b = int(d.length.argmax())
        dspark.cache_fork(d.c, d.seq[b:b + 1], ints([0]), ints([n]))
        at = torch.arange(n, device="cuda")
        for plane in range(4):
            pool = d.c.pool.view(4, *d.c.pool.shape[2:])[plane]
            rows = [pool[d.c.block_table[s].long()[at // 16], :, at % 16]
                    for s in (0, int(d.seq[b]))]
            assert torch.equal(rows[0], rows[1])
        assert dspark.read_device_error(d.c) == 0


@pytest.mark.parametrize("dtype", [BF, F32])
def test_a_line_of_tiles_beyond_32_bits_is_refused(cuda, dtype):
    kv, page = 64, 4096
    c = dspark.PagedCache(1, 1, page, kv, 64, 16, 1 << 18, dtype=dtype)
    c.block_table.zero_()
    c.page_count.fill_(1 << 18)
    q = torch.ones(16, 1, kv, 64, dtype=dtype, device="cuda")
    out = torch.full_like(q, 5.0)
    length = ints([(1 << 30) - 1] * 16)
    dspark.tree_attention(c, 0, q, length, out=out)
    assert (out == 5).all()
    assert dspark.read_device_error(c) == 7


@pytest.mark.parametrize("dtype,T", [(BF, 2), (F32, 3)])
def test_the_largest_batch(cuda, dtype, T):
    """1024 sequences give the same bits as the same ones 64 at a time, where
    no unit is cut, or nearly so."""
    B, kv, D, page = 1024, 1, 64, 16
    g = torch.Generator(device="cuda").manual_seed(9)
    c = dspark.PagedCache(1, 6000, page, kv, D, B, 8, dtype=dtype)
    length = torch.randint(0, 70, (B,), generator=g, device="cuda").int()
    count = torch.randint(0, T + 1, (B,), generator=g, device="cuda").int()
    dspark.cache_reserve(c, length, T)
    c.pool.normal_(generator=g)
    q = torch.randn(B, T, 2, D, generator=g, device="cuda").to(dtype)
    out, lse = dspark.tree_attention(c, 0, q, length, token_count=count, with_lse=True)
    # Of each of the two: weights and output rounded to bfloat16 (2^-8 each), or
    # some 75 sums, an exponential of 2^-22 and an exponent below 64 in float32
    # (75 + 4 + 64 times 2^-24, below 2^-16).
    size = float(c.pool.float().abs().max())
    tol = size * (2 * (2 * 2.0 ** -8 + 2.0 ** -16) if dtype == BF else 2 * 2.0 ** -16)
    for b in range(0, B, 64):
        seq = torch.arange(b, b + 64, dtype=torch.int32, device="cuda")
        o, l = dspark.tree_attention(c, 0, q[b:b + 64], length[b:b + 64], seq=seq,
                                     token_count=count[b:b + 64], with_lse=True)
        for i, n in enumerate(count[b:b + 64].tolist()):
            assert ((o[i, :n].float() - out[b + i, :n].float()).abs() <= tol).all()
            assert ((l[i, :n] - lse[b + i, :n]).abs() <= 2.0 ** -15).all()
    assert dspark.read_device_error(c) == 0


def test_long_lists_of_shared_pages(cuda):
    """More pages in a call than a block takes in one pass: shared by many,
    given up in two calls, and a row that is named twice counts once."""
    page, n = 4, 90
    c = dspark.PagedCache(1, 400, page, 1, 8, 70, 100)
    m = PageModel(400, page, 70, 100)
    dspark.cache_reserve(c, ints([0]), n * page + 1)
    m.reserve([0], [0], n * page + 1)
    kids = list(range(1, 61))
    dspark.cache_fork(c, ints([0] * 60), ints(kids), ints([n * page + 1] * 60))
    m.fork([0] * 60, kids, [n * page + 1] * 60)
    m.check(c)
    dspark.cache_release(c, ints(kids[5:]))
    m.release(kids[5:])
    m.check(c)
    dspark.cache_release(c, ints(kids[:5] + [0]))
    m.release(kids[:5] + [0])
    m.check(c)
    assert int(c.control[1]) == 400
    # all in one call, more than 4096 entries
    dspark.cache_reserve(c, ints([0]), n * page)
    m.reserve([0], [0], n * page)
    dspark.cache_fork(c, ints([0] * 60), ints(kids), ints([n * page] * 60))
    m.fork([0] * 60, kids, [n * page] * 60)
    dspark.cache_release(c, ints([0] + kids))
    m.release([0] + kids)
    m.check(c)
    dspark.cache_reserve(c, ints([0, 0]), 9, seq=ints([3, 5]))
    dspark.cache_release(c, ints([3, 5, 3]))
    assert int(c.control[1]) == 400
    assert sorted(c.free_list.tolist()) == list(range(400))
    assert (c.ref_count == 0).all()


def test_append_refuses_uneven_tokens(cuda):
    d = Decoder(BF)
    x = torch.zeros(4, 9, 6, 64, dtype=BF, device="cuda")
    a = dict(position=d.position, cos_sin=d.cs, seq=d.seq)
    k = torch.zeros(3, 8, 2, 64, dtype=BF, device="cuda")
    for q in (x[:3, :8],                     # a gap between sequences
              x.transpose(2, 3)[:3, :8],     # heads inside
              x[:3, :8].transpose(0, 1)[:3]):
        with pytest.raises(ValueError):
            dspark.cache_append(d.c, 0, q, k, k, d.length, **a)
    with pytest.raises(ValueError):
        dspark.cache_append(d.c, 0, x[:3, :8].contiguous(), k.expand(3, 8, 2, 64)[:, :, :, :32], k,
                            d.length, **a)


def test_attention_refuses_to_work_in_place(cuda):
    d = Decoder(BF)
    with pytest.raises(dspark.DsparkError):
        dspark.tree_attention(d.c, 0, d.q[0], d.length, out=d.q[0])
