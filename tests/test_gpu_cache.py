"""The paged cache on the GPU: its bookkeeping against a list model, copies and
moves bit for bit, and the normalisation and rotation against 64 bits."""
import numpy as np
import pytest
import torch

import ancestral_draft_sampling_gb300 as dspark
from tests.cache_ref import PageModel, place, rotate

pytestmark = pytest.mark.gpu


def ints(x):
    return torch.tensor(x, dtype=torch.int32, device="cuda")


def make(page=16, num_pages=64, max_seqs=8, max_pages=16, layers=2, kv_heads=2, dim=64,
         dtype=torch.bfloat16, seed=0):
    c = dspark.PagedCache(layers, num_pages, page, kv_heads, dim, max_seqs, max_pages, dtype=dtype)
    g = torch.Generator(device="cuda").manual_seed(seed)
    c.pool.normal_(generator=g)
    return c, PageModel(num_pages, page, max_seqs, max_pages)


def error(c):
    return dspark.read_device_error(c)


def test_new_cache_is_empty(cuda):
    c, m = make()
    m.check(c)
    assert error(c) == 0


@pytest.mark.parametrize("page,max_seqs,seed", [(1, 5, 0), (16, 8, 1), (64, 40, 2), (7, 1000, 3)])
def test_bookkeeping_follows_the_model(cuda, page, max_seqs, seed):
    """Random calls, shared pages among them: tables, counts, holds and the
    stack's order are the model's after every one."""
    rng = np.random.default_rng(seed)
    num_pages = 4 * max_seqs + 40
    c, m = make(page=page, num_pages=num_pages, max_seqs=max_seqs, max_pages=60, layers=1,
                kv_heads=1, dim=8)
    length = [0] * max_seqs
    for _ in range(25):
        B = int(rng.integers(1, max_seqs + 1))
        seq = rng.permutation(max_seqs)[:B].tolist()
        n = [length[s] for s in seq]
        op = rng.integers(0, 4)
        if op <= 1:
            T = int(rng.integers(1, 3 * page + 2))
            dspark.cache_reserve(c, ints(n), T, seq=ints(seq))
            m.reserve(seq, n, T)
            m.check(c)
            # keep what fits the pages that the sequence got
            acc = [int(rng.integers(-1, T)) for _ in seq]
            keep = [0 if a < 0 else a + 1 for a in acc]
            keep = [k if x + k <= len(m.held[s]) * page else 0 for s, x, k in zip(seq, n, keep)]
            acc = [k - 1 if k else -1 for k in keep]
            got = dspark.cache_accept(c, ints(n), ints(acc), T, seq=ints(seq))
            now = m.accept(seq, n, keep)
            assert got.tolist() == now
            for s, x in zip(seq, now):
                length[s] = x
        elif op == 2 and max_seqs > 1:
            half = max(1, B // 2)
            kids = seq[:half] if half < B else seq[:1]
            rest = [s for s in range(max_seqs) if s not in kids]
            par = [rest[int(rng.integers(0, len(rest)))] for _ in kids]
            cut = [int(rng.integers(0, length[p] + 1)) for p in par]
            before = c.pool.clone()
            dspark.cache_fork(c, ints(par), ints(kids), ints(cut))
            copies = m.fork(par, kids, cut)
            for a, b, rows in copies:
                before[:, :, b, :, :rows] = before[:, :, a, :, :rows]
            assert torch.equal(before, c.pool)
            for s, x in zip(kids, cut):
                length[s] = x if len(m.held[s]) * page >= x else 0
        else:
            dspark.cache_release(c, ints(seq))
            m.release(seq)
            for s in seq:
                length[s] = 0
        m.check(c)
    assert error(c) in (0, m.error) or m.error == 8


def test_reserve_and_release_leave_the_stack_as_it_was(cuda):
    c, m = make(num_pages=50)
    before = c.free_list.clone()
    dspark.cache_reserve(c, ints([3, 40, 0]), 20, seq=ints([5, 1, 2]))
    dspark.cache_release(c, ints([5, 1, 2]))
    assert torch.equal(before, c.free_list)
    m.check(c)


def test_reserve_runs_out(cuda):
    """Those that do not fit get nothing, the others are served."""
    c, m = make(num_pages=10, max_seqs=4, page=16)
    args = [0, 0, 0], 64, [0, 1, 2]
    dspark.cache_reserve(c, ints(args[0]), args[1], seq=ints(args[2]))
    m.reserve(args[2], args[0], args[1])
    m.check(c)
    assert error(c) == 8 and error(c) == 0
    dspark.cache_reserve(c, ints([0, 0]), 17, seq=ints([2, 3]))  # two are left
    m.reserve([2, 3], [0, 0], 17)
    m.check(c)
    assert error(c) == 8
    c2, m2 = make(max_pages=3, num_pages=20, max_seqs=2, page=16)
    dspark.cache_reserve(c2, ints([40, 48]), 1)  # 48 + 1 tokens: four pages
    m2.reserve([0, 1], [40, 48], 1)
    m2.check(c2)
    assert error(c2) == 8


def test_sequences_out_of_range_are_skipped(cuda):
    c, m = make(max_seqs=3)
    dspark.cache_reserve(c, ints([5, 5, 5, -1]), 9, seq=ints([0, 3, -1, 1]))
    m.reserve([0, 3, -1, 1], [5, 5, 5, -1], 9)
    m.check(c)
    assert error(c) in (6, 7)
    got = dspark.cache_accept(c, ints([5, 5]), ints([2, 2]), 9, seq=ints([7, 0]))
    assert got.tolist() == [5, 8] and error(c) == 6
    m.accept([0], [5], [3])
    m.check(c)
    dspark.cache_release(c, ints([9, 0]))
    m.release([0])
    m.check(c)
    assert error(c) == 6


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("page,paths", [
    (16, [[0, 2, 3, 5, 9], [0, 1, 2, 3, 4], [2, 3, 4, 5, 6], [0, 1, 2, 10, 11]]),
    (4, [[1, 2, 3, 4, 5], [0, 5, 9, 10, 11], [7, 8, 9, 10, 11], [0, 1, 3, 4, 11]]),
    (1, [[3, 4, 6, 7, 8], [0, 1, 2, 3, 9], [0, 2, 4, 6, 8], [0, 9, 10, 11, 11]]),
])
def test_accept_moves_the_path(cuda, page, paths, dtype):
    """Overlapping moves, every page size, and a path that is none (it keeps
    nothing)."""
    T, length, accepted = 12, [0, 7, 33, 18], [3, 4, 2, 4]
    c, m = make(page=page, num_pages=300, max_pages=200, dtype=dtype, layers=3)
    dspark.cache_reserve(c, ints(length), T)
    m.reserve(range(4), length, T)
    want = c.pool.clone()
    keep = []
    for b, p in enumerate(paths):
        n = accepted[b] + 1
        if any(y <= x for x, y in zip(p, p[1:n])):
            keep.append(0)
            continue
        keep.append(n)
        ids, slots = place(c, b, length[b] + T)
        src = torch.tensor([length[b] + x for x in p[:n]])
        dst = torch.arange(length[b], length[b] + n)
        want[:, :, ids[dst].cuda(), :, slots[dst].cuda()] = want[:, :, ids[src].cuda(), :, slots[src].cuda()]
    new = torch.full((4,), -7, dtype=torch.int32, device="cuda")
    got = dspark.cache_accept(c, ints(length), ints(accepted), T, path=ints(paths), new_length=new)
    assert got is new and new.tolist() == m.accept(range(4), length, keep)
    assert torch.equal(c.pool, want)
    m.check(c)
    assert error(c) == (9 if 0 in keep else 0)


def test_accept_of_a_wide_tree_in_place(cuda):
    """64 nodes, 64 kept ones, and lengths updated where they lie."""
    T = 64
    c, m = make(page=32, num_pages=64, layers=1, kv_heads=3, dim=40)
    length = ints([5, 70])
    dspark.cache_reserve(c, length, T)
    m.reserve([0, 1], [5, 70], T)
    want = c.pool.clone()
    path = torch.arange(T, dtype=torch.int32, device="cuda").repeat(2, 1)
    path[1, :32] = torch.arange(1, 64, 2)
    ids, slots = place(c, 1, 70 + T)
    src, dst = torch.arange(71, 134, 2), torch.arange(70, 102)
    want[:, :, ids[dst].cuda(), :, slots[dst].cuda()] = want[:, :, ids[src].cuda(), :, slots[src].cuda()]
    dspark.cache_accept(c, length, ints([63, 31]), T, path=path, new_length=length)
    m.accept([0, 1], [5, 70], [64, 32])
    assert length.tolist() == [69, 102] and torch.equal(c.pool, want)
    m.check(c)


@pytest.mark.parametrize("accepted,path,extra,code", [
    ([-1], None, 1, 0), ([4], None, 1, 9), ([0], None, 5, 9), ([3], None, 1, 0),
    ([2], [[0, 2, 5, 3]], 1, 9), ([3], [[0, 1, 2]], 1, 9), ([1], [[-1, 2]], 1, 9),
    ([-2147483648], [[0, 1]], 1, 0), ([2147483647], [[0, 1]], 1, 9), ([0], None, 0, 0),
])
def test_accept_of_none_and_bad_paths(cuda, accepted, path, extra, code):
    c, m = make()
    dspark.cache_reserve(c, ints([30]), 4)
    m.reserve([0], [30], 4)
    before = c.pool.clone()
    got = dspark.cache_accept(c, ints([30]), ints(accepted), 4, extra=extra,
                              path=ints(path) if path else None)
    keep = 0 if code or accepted[0] < 0 else accepted[0] + extra
    assert got.tolist() == m.accept([0], [30], [keep]) and error(c) == code
    assert torch.equal(before, c.pool)
    m.check(c)


def test_fork_shares_copies_and_refuses(cuda):
    c, m = make(page=16, num_pages=12, layers=3)
    dspark.cache_reserve(c, ints([0, 0]), 40)
    m.reserve([0, 1], [0, 0], 40)
    want = c.pool.clone()
    # three children of one parent: at a page's end, inside one, and empty
    dspark.cache_fork(c, ints([0, 0, 0, 1]), ints([2, 3, 4, 5]), ints([32, 33, 0, 40]))
    for a, b, rows in m.fork([0, 0, 0, 1], [2, 3, 4, 5], [32, 33, 0, 40]):
        want[:, :, b, :, :rows] = want[:, :, a, :, :rows]
    assert torch.equal(want, c.pool)
    m.check(c)
    # again: the children's earlier pages go back first
    dspark.cache_fork(c, ints([1, 0]), ints([3, 2]), ints([35, 47]))
    for a, b, rows in m.fork([1, 0], [3, 2], [35, 47]):
        want[:, :, b, :, :rows] = want[:, :, a, :, :rows]
    assert torch.equal(want, c.pool) and error(c) == 0
    m.check(c)
    # the parent's pages stay while a child holds them
    dspark.cache_release(c, ints([0, 1]))
    m.release([0, 1])
    m.check(c)
    for par, kid in (([2, 3], [3, 6]), ([2, 2], [6, 6]), ([2], [2])):
        dspark.cache_fork(c, ints(par), ints(kid), ints([1] * len(par)))
        m.fork(par, kid, [1] * len(par))
        m.check(c)
        assert error(c) == 11
    dspark.cache_fork(c, ints([2, 2]), ints([6, 7]), ints([49, 5]))  # more than it holds
    m.fork([2, 2], [6, 7], [49, 5])
    m.check(c)
    assert error(c) == 7
    free = int(c.control[1])
    dspark.cache_reserve(c, ints([0]), 16 * free, seq=ints([0]))
    m.reserve([0], [0], 16 * free)
    dspark.cache_fork(c, ints([2, 2]), ints([6, 5]), ints([5, 32]))
    m.fork([2, 2], [6, 5], [5, 32])
    m.check(c)
    error(c)


def test_release_of_pages_shared_by_all(cuda):
    """Children give up one parent's pages in one call: each goes back once."""
    c, m = make(page=4, num_pages=40)
    dspark.cache_reserve(c, ints([0]), 26)
    m.reserve([0], [0], 26)
    dspark.cache_fork(c, ints([0] * 4), ints([1, 2, 3, 4]), ints([26, 24, 11, 5]))
    m.fork([0] * 4, [1, 2, 3, 4], [26, 24, 11, 5])
    dspark.cache_release(c, ints([0, 3]))
    m.release([0, 3])
    m.check(c)
    dspark.cache_release(c, ints([4, 2, 1]))
    m.release([4, 2, 1])
    m.check(c)
    assert int(c.control[1]) == 40


def test_corrupt_tables_are_not_followed(cuda):
    c, _ = make(page=16, num_pages=12)
    dspark.cache_reserve(c, ints([0, 0]), 30)
    c.block_table[0, 1] = 12
    c.block_table[1, 0] = -5
    pool = c.pool.clone()
    dspark.cache_accept(c, ints([10, 10]), ints([4, 4]), 20, path=ints([[0, 1, 2, 12, 15]] * 2))
    assert error(c) == 7 and torch.equal(pool, c.pool)
    dspark.cache_release(c, ints([0, 1]))
    assert error(c) == 7
    c.control[1] = 1000
    dspark.cache_release(c, ints([0]))
    assert int(c.control[1]) <= 12


# ------------------------------------------------------------------ append
def append_bound(size, D, dtype):
    """One rounding of the result (2^-8 of it in bfloat16, 2^-24 in float32)
    after a float32 mean of D squares, its root, three products and a sum:
    (D / 2 + 16) 2^-24 of the magnitudes that a value is made of."""
    u = 2.0 ** -24
    bound = (D / 2 + 16) * u * size
    return bound + (2.0 ** -8 if dtype == torch.bfloat16 else u) * (size + bound)


CASES = [  # dtype, D, rot, interleaved, norm, heads, kv_heads, page, T
    (torch.bfloat16, 128, 128, False, True, 8, 2, 64, 8),
    (torch.bfloat16, 128, 64, True, True, 4, 4, 16, 1),
    (torch.bfloat16, 64, 32, False, False, 6, 2, 32, 5),
    (torch.bfloat16, 64, 36, False, True, 3, 1, 7, 9),     # halves end inside a lane
    (torch.bfloat16, 96, 96, True, True, 5, 5, 16, 3),     # no power of two
    (torch.bfloat16, 40, 8, False, True, 2, 1, 1, 4),
    (torch.bfloat16, 256, 256, False, True, 4, 2, 128, 2),
    (torch.bfloat16, 8, 2, True, True, 32, 1, 16, 6),
    (torch.float32, 128, 128, False, True, 4, 2, 16, 7),
    (torch.float32, 64, 20, True, False, 3, 3, 8, 2),
    (torch.float32, 256, 128, False, True, 2, 1, 16, 3),
    (torch.float32, 128, 6, False, True, 2, 2, 16, 64),
]


@pytest.mark.parametrize("dtype,D,rot,inter,norm,heads,kv,page,T", CASES)
@pytest.mark.parametrize("parts", [False, True])
def test_append(cuda, dtype, D, rot, inter, norm, heads, kv, page, T, parts):
    """Separate tensors and parts of one projection, sequences in any order,
    fewer tokens than T: results within the roundings, everything else as it
    was."""
    g = torch.Generator(device="cuda").manual_seed(D + T)
    B, length, count, seq = 3, [0, 21, 5], [T, max(1, T - 1), 0], [4, 0, 2]
    c, _ = make(page=page, num_pages=500, max_pages=200, kv_heads=kv, dim=D, dtype=dtype)
    dspark.cache_reserve(c, ints(length), T, seq=ints(seq))

    def normal(*shape):
        return torch.randn(*shape, generator=g, device="cuda").to(dtype)
    if parts:
        qkv = normal(B, T, heads + 2 * kv, D)
        q, k, v = qkv[:, :, :heads], qkv[:, :, heads:heads + kv], qkv[:, :, heads + kv:]
    else:
        q, k, v = normal(B, T, heads, D), normal(B, T, kv, D), normal(B, T, kv, D)
    cos_sin = torch.randn(90, rot, generator=g, device="cuda")
    position = torch.randint(0, 90, (B, T), generator=g, device="cuda", dtype=torch.int32)
    wq = torch.randn(D, generator=g, device="cuda") if norm else None
    wk = torch.randn(D, generator=g, device="cuda") if norm else None
    out = torch.full((B, T, heads, D), 7.0, dtype=dtype, device="cuda")
    want = c.pool.double().cpu()
    size = torch.zeros_like(want)
    rq, sq = rotate(q.cpu(), None if wq is None else wq.cpu(), 1e-5, cos_sin.cpu(), position.cpu(), inter)
    rk, sk = rotate(k.cpu(), None if wk is None else wk.cpu(), 1e-5, cos_sin.cpu(), position.cpu(), inter)
    for b in range(B):
        ids, slots = place(c, seq[b], length[b] + T)
        for t in range(count[b]):
            i = length[b] + t
            want[1, 0, ids[i], :, slots[i]] = rk[b, t]
            size[1, 0, ids[i], :, slots[i]] = append_bound(sk[b, t], D, dtype)
            want[1, 1, ids[i], :, slots[i]] = v[b, t].double().cpu()
        rq[b, count[b]:] = 7.0
        sq[b, count[b]:] = 0.0
    got = dspark.cache_append(c, 1, q, k, v, ints(length), position=position, cos_sin=cos_sin,
                              q_weight=wq, k_weight=wk, eps=1e-5, interleaved=inter,
                              token_count=ints(count), seq=ints(seq), q_out=out)
    assert got is out and error(c) == 0
    assert ((out.double().cpu() - rq).abs() <= append_bound(sq, D, dtype) * (sq > 0)).all()
    assert ((c.pool.double().cpu() - want).abs() <= size).all()


def test_append_in_place_and_many_tokens(cuda):
    """q_out may be q; a prompt's tokens take the kernel's wide form and give
    what a token at a time gives."""
    c, _ = make(page=64, num_pages=300, max_pages=100, kv_heads=8, dim=128, layers=1)
    B, T = 2, 3001
    dspark.cache_reserve(c, ints([0, 10]), T)
    g = torch.Generator(device="cuda").manual_seed(5)
    qkv = torch.randn(B, T, 48, 128, generator=g, device="cuda").bfloat16()
    q, k, v = qkv[:, :, :32].contiguous(), qkv[:, :, 32:40], qkv[:, :, 40:]
    pos = torch.arange(T, dtype=torch.int32, device="cuda").repeat(2, 1)
    cs = torch.randn(T, 128, generator=g, device="cuda")
    w = torch.randn(128, generator=g, device="cuda")
    args = dict(cos_sin=cs, q_weight=w, k_weight=w)
    all_at_once = dspark.cache_append(c, 0, q, k, v, ints([0, 10]), position=pos, **args)
    pool = c.pool.clone()
    for t in (0, 1, 1500, 3000):
        one = dspark.cache_append(c, 0, q[:, t:t + 1], k[:, t:t + 1], v[:, t:t + 1], ints([t, 10 + t]),
                                  position=pos[:, t:t + 1].contiguous(), **args)
        assert torch.equal(one, all_at_once[:, t:t + 1])
    assert torch.equal(pool, c.pool)
    dspark.cache_append(c, 0, q, k, v, ints([0, 10]), position=pos, q_out=q, **args)
    assert torch.equal(q, all_at_once) and torch.equal(pool, c.pool) and error(c) == 0


def test_append_refuses_places_and_positions_on_the_device(cuda):
    c, _ = make(page=16, num_pages=20, kv_heads=1, dim=64, layers=1)
    dspark.cache_reserve(c, ints([0, 0]), 16)
    q = torch.randn(2, 2, 2, 64, device="cuda").bfloat16()
    kv = torch.randn(2, 2, 1, 64, device="cuda").bfloat16()
    cs = torch.randn(8, 64, device="cuda")
    pool = c.pool.clone()
    pos = ints([[0, 1], [2, 3]])
    # behind the held pages, before the start: queries only
    for bad in ([16, 40], [-1, -2147483648], [2147483646, 15]):
        before = c.pool.clone()
        a = dspark.cache_append(c, 0, q, kv, kv, ints(bad), position=pos, cos_sin=cs)
        assert error(c) == 7
        if bad[1] != 15 and bad[0] != -1:
            assert torch.equal(before, c.pool)
    b = dspark.cache_append(c, 0, q, kv, kv, ints([0, 0]), position=pos, cos_sin=cs)
    assert torch.equal(a, b) and error(c) == 0
    # positions outside the table: not rotated
    out = dspark.cache_append(c, 0, q, kv, kv, ints([0, 0]), position=ints([[-1, 8], [2, 3]]), cos_sin=cs)
    assert error(c) == 10
    assert torch.equal(out[0], q[0]) and torch.equal(out[1], b[1])
    out = torch.zeros_like(q)
    dspark.cache_append(c, 0, q, kv, kv, ints([0, 0]), position=pos, cos_sin=cs, seq=ints([8, 1]), q_out=out)
    assert error(c) == 6 and not out[0].any() and torch.equal(out[1], b[1])
    assert pool.shape == c.pool.shape


def test_append_keeps_infinities_where_they_are(cuda):
    """Dims behind the rotated ones keep their bits; without a norm an
    infinity stays in its pair."""
    c, _ = make(page=16, kv_heads=1, dim=64, layers=1)
    dspark.cache_reserve(c, ints([0]), 1)
    q = torch.ones(1, 1, 1, 64, device="cuda").bfloat16()
    q[..., 40], q[..., 3] = float("inf"), float("nan")
    cs = torch.cat([torch.ones(4, 16), torch.zeros(4, 16)], 1).cuda()
    out = dspark.cache_append(c, 0, q, q, q, ints([0]), position=ints([[1]]), cos_sin=cs)[0, 0, 0].float()
    assert out[40] == float("inf") and torch.isnan(out[3])
    others = [i for i in range(64) if i not in (40, 3, 19)]
    assert (out[others] == 1).all()
