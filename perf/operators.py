"""The paged key/value cache of speculative decoding and the attention that
reads it, as cases to be timed and compared.

A decoding step around the draft block: room for the drafted tokens is
reserved in the cache, each layer normalises and rotates their queries and
keys and stores keys and values (``append``), attends from the drafted tree
over the cache (``attend``), and after verification the accepted path is moved
together and the pages behind it are freed (``accept``).  A prompt shared by
several requests is forked (``fork``).

Where ``own`` is false, ``run`` computes the operators from elementary torch
operations in 32 bits; where it is true, it calls the framework.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELT = {"bf16": 2, "f32": 4}


def listed():
    return [
        # One request at the start of its answer: the last token and seven
        # drafts are verified.  Latency counts.
        dict(name="attend one request", op="attend", dtype="bf16", batch=1, tokens=8, kv_heads=8, group=4, dim=128,
             page=64, longest=1000, mask="causal", window=0, ragged=False),
        # Single tokens (no drafts) of a batch, small heads and pages, a
        # sliding window.
        dict(name="attend single tokens", op="attend", dtype="bf16", batch=44, tokens=1, kv_heads=8, group=8, dim=64,
             page=16, longest=8200, mask="causal", window=4096, ragged=False),
        # The full serving batch with seven drafts each and long contexts;
        # the last rows of some requests are padding.
        dict(name="attend full batch", op="attend", dtype="bf16", batch=88, tokens=8, kv_heads=8, group=4, dim=128,
             page=64, longest=16000, mask="causal", window=0, ragged=True),
        # A wide tree of drafts: many query rows for each key.
        dict(name="attend wide tree", op="attend", dtype="bf16", batch=8, tokens=61, kv_heads=8, group=8, dim=128,
             page=32, longest=5000, mask="tree", window=0, ragged=False),
        # A float32 drafter's block, which sees itself whole.
        dict(name="attend block f32", op="attend", dtype="f32", batch=3, tokens=7, kv_heads=2, group=3, dim=64,
             page=16, longest=777, mask="full", window=0, ragged=True),
        # One token of one request.
        dict(name="append one token", op="append", dtype="bf16", batch=1, tokens=1, kv_heads=8, group=4, dim=128,
             page=64, longest=1000, rot=128, norm=True, interleaved=False, ragged=False),
        # The drafted tokens of the full batch.
        dict(name="append full batch", op="append", dtype="bf16", batch=88, tokens=8, kv_heads=8, group=4, dim=128,
             page=64, longest=16000, rot=128, norm=True, interleaved=False, ragged=True),
        # Two prompts, half of each head rotated in neighbouring pairs.
        dict(name="append prompts", op="append", dtype="bf16", batch=2, tokens=8191, kv_heads=8, group=4, dim=128,
             page=64, longest=77, rot=64, norm=True, interleaved=True, ragged=True),
        # The drafter's own five-layer cache after a step of the full batch.
        dict(name="accept full batch", op="accept", dtype="bf16", batch=88, tokens=8, kv_heads=8, dim=128, page=64,
             longest=500, layers=5),
        # A wide tree's accepted path in every layer of a target model.
        dict(name="accept wide tree", op="accept", dtype="bf16", batch=8, tokens=61, kv_heads=8, dim=128, page=32,
             longest=900, layers=32),
        # Two answers to one short prompt.
        dict(name="fork pair", op="fork", dtype="bf16", parents=1, children=2, kv_heads=8, dim=128, page=64,
             longest=210, layers=5),
        # Sixteen answers each to four long prompts.
        dict(name="fork many", op="fork", dtype="bf16", parents=4, children=64, kv_heads=8, dim=128, page=64,
             longest=4000, layers=16),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["attend", "attend", "attend", "append", "accept", "fork"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim, page = rng.choice([64, 128]), rng.choice([16, 32, 64, 128])
    kv = rng.choice([1, 2, 3, 4, 8, 16])
    if op == "attend":
        group, batch, tokens = rng.randint(1, 8), _spread(rng, 1, 88), _spread(rng, 1, 64)
        most = 88 * 16000 * 8 * 128 // (4 if dtype == "bf16" else 64)  # keys times heads times dim
        longest = max(32, min(_spread(rng, 64, 16000), most // (batch * kv * dim)))
        rows = 150_000_000 // (batch * kv * longest)  # scores that the plain form holds, over heads
        tokens = max(1, min(tokens, rows // group, 256 // group if longest > 4000 else 64))
        mask = rng.choice(["causal", "tree", "full"])
        return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, kv_heads=kv, group=group, dim=dim, page=page,
                    longest=longest, mask=mask, window=rng.choice([0, 0, _spread(rng, 100, 4096)]),
                    ragged=rng.random() < 0.5)
    if op == "append":
        group, batch = rng.randint(1, 8), _spread(rng, 1, 88)
        tokens = min(_spread(rng, 1, 8191), max(1, 16000 * 40 // (batch * kv * (group + 2) * (2 if dtype == "f32" else 1))))
        return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, kv_heads=kv, group=group, dim=dim, page=page,
                    longest=_spread(rng, 1, 1000), rot=rng.choice([dim, dim // 2]), norm=rng.random() < 0.7,
                    interleaved=rng.random() < 0.5, ragged=rng.random() < 0.5)
    layers = rng.randint(1, 16)
    if op == "accept":
        return dict(op=op, dtype=dtype, batch=_spread(rng, 1, 88), tokens=_spread(rng, 2, 64), kv_heads=min(kv, 8),
                    dim=dim, page=page, longest=_spread(rng, 16, 500), layers=min(layers, 5))
    parents = rng.randint(1, 4)
    return dict(op=op, dtype=dtype, parents=parents, children=parents * rng.randint(1, 8), kv_heads=min(kv, 8),
                dim=dim, page=page, longest=_spread(rng, 16, 2000), layers=layers)


# ------------------------------------------------------------ the sizes
def _lengths(case, n):
    """Committed lengths: from a quarter of the longest to the longest, one
    request without any where the batch is ragged."""
    top = case["longest"]
    got = [top if b == 0 else max(1, int(top * (0.25 + 0.75 * ((b * 0.6180339887498949) % 1.0)))) for b in range(n)]
    if case.get("ragged") and n > 2:
        got[n // 2] = 0
    return got


def _counts(case):
    """Drafted tokens of each request: all of them, or from one up."""
    B, T = case["batch"], case["tokens"]
    if not case.get("ragged"):
        return [T] * B
    return [T if b == 0 else 1 + int(T * ((b * 0.6180339887498949) % 1.0)) for b in range(B)]


def _accepted(case):
    """Accepted drafts of each request: none to all of a path."""
    return [(b * 3 + 2) % _path_width(case["tokens"]) for b in range(case["batch"])]


def _path_width(tokens):
    """Nodes of an accepted path, the root among them: eight at most, and
    few enough that the kept rows end before the path's later nodes begin
    (so a second pass finds the rows that the first one found)."""
    return min(8, (tokens + 1) // 2)


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------ the inputs
def _cache(case, held, rows, spare, gen, layers):
    """A pool whose sequences hold held[i] pages each, scattered at random,
    as tensors: what a program's cache consists of."""
    device = "cuda"
    total = sum(held)
    num_pages, max_pages = total + spare, max(held) + 6
    order = torch.randperm(num_pages, generator=gen, device=device).to(torch.int32)
    starts = torch.tensor([sum(held[:i]) for i in range(rows)], device=device)
    have = torch.tensor(held, device=device)
    j = torch.arange(max_pages, device=device)[None]
    table = torch.where(j < have[:, None], order[(starts[:, None] + j).clamp(max=num_pages - 1)], -1).to(torch.int32)
    ref = torch.zeros(num_pages, dtype=torch.int32, device=device)
    ref[order[:total].long()] = 1
    free = torch.full((num_pages,), -1, dtype=torch.int32, device=device)
    free[:spare] = order[total:]
    control = torch.zeros(64 + 2 * 1024, dtype=torch.int32, device=device)
    control[1] = spare
    dtype = DTYPES[case["dtype"]]
    pool = torch.empty(layers, 2, num_pages, case["kv_heads"], case["page"], case["dim"], dtype=dtype, device=device)
    pool.normal_(generator=gen)
    state = dict(pool=pool, table=table.contiguous(), count=have.to(torch.int32), ref=ref, free=free, control=control)
    if own:  # the handle that a program keeps: it names the tensors and holds no data
        import ancestral_draft_sampling_gb300 as dspark
        state["cache"] = dspark.PagedCache.from_tensors(pool, state["table"], state["count"], ref, free, control)
    return state


def _masks(case, gen):
    """For each drafted token the drafted tokens that it sees (bit j: token
    j), and its depth."""
    B, T = case["batch"], case["tokens"]
    one = torch.ones(B, T, dtype=torch.int64, device="cuda")
    t = torch.arange(T, device="cuda")
    if case["mask"] == "full":
        return torch.full_like(one, -1 if T == 64 else (1 << T) - 1), t[None].expand(B, T)
    if case["mask"] == "causal":
        return torch.where(t == 63, -1, (one << ((t + 1) % 64)) - 1), t[None].expand(B, T)
    mask, depth = one.clone(), torch.zeros_like(one)
    parents = (torch.rand(B, T, generator=gen, device="cuda") * t).long()
    rows = torch.arange(B, device="cuda")
    for i in range(1, T):
        mask[:, i] = mask[rows, parents[:, i]] | (one[:, i] << i)
        depth[:, i] = depth[rows, parents[:, i]] + 1
    return mask, depth


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype, page = case["op"], DTYPES[case["dtype"]], case["page"]
    i32 = dict(dtype=torch.int32, device="cuda")

    def normal(*shape):
        return torch.randn(*shape, generator=gen, device="cuda").to(dtype)

    if op == "fork":
        P, C = case["parents"], case["children"]
        lens = _lengths(case, P)
        held = [_pages(n, page) for n in lens] + [0] * C
        s = _cache(case, held, P + C, C + 3, gen, case["layers"])
        parent = torch.arange(C, **i32) % P
        s |= dict(case=case, parent=parent, child=torch.arange(C, **i32) + P,
                  length=torch.tensor(lens, **i32)[parent.long()].contiguous())
        return s
    B, T = case["batch"], case["tokens"]
    lens = _lengths(case, B)
    length = torch.tensor(lens, **i32)
    if op == "accept":
        held = [_pages(n, page) for n in lens]
        s = _cache(case, held, B, B * (_pages(T, page) + 1), gen, case["layers"])
        accepted = torch.tensor(_accepted(case), **i32)
        # the accepted path: the root, then ever later nodes behind the kept rows
        width = _path_width(T)
        later = torch.rand(B, T, generator=gen, device="cuda")
        later[:, :width] = 2.0
        path = later.argsort(dim=1)[:, :width - 1].sort(dim=1).values
        path = torch.cat([torch.zeros(B, 1, dtype=path.dtype, device="cuda"), path], dim=1)
        path = path.to(torch.int32).contiguous()
        s |= dict(case=case, length=length, accepted=accepted, path=path, new_length=torch.zeros(B, **i32))
        return s
    Hq, Hkv, D = case["kv_heads"] * case["group"], case["kv_heads"], case["dim"]
    held = [_pages(n + T, page) for n in lens]
    s = _cache(case, held, B, 3, gen, 1)
    counts = torch.tensor(_counts(case), **i32)
    s |= dict(case=case, length=length, counts=counts if case["ragged"] else None)
    if op == "append":
        # one projection's output: queries, keys and values of a token side by side
        qkv = normal(B, T, Hq + 2 * Hkv, D)
        top = max(lens) + T
        freq = 10000.0 ** (-torch.arange(case["rot"] // 2, dtype=torch.float64, device="cuda") * 2 / case["rot"])
        angle = torch.arange(top, dtype=torch.float64, device="cuda")[:, None] * freq
        s |= dict(q=qkv[:, :, :Hq], k=qkv[:, :, Hq:Hq + Hkv], v=qkv[:, :, Hq + Hkv:],
                  cos_sin=torch.cat([angle.cos(), angle.sin()], dim=1).float().contiguous(),
                  position=(length[:, None] + torch.arange(T, **i32)[None]).contiguous(),
                  wq=1 + 0.1 * torch.randn(D, generator=gen, device="cuda") if case["norm"] else None,
                  wk=1 + 0.1 * torch.randn(D, generator=gen, device="cuda") if case["norm"] else None,
                  q_out=torch.zeros(B, T, Hq, D, dtype=dtype, device="cuda"))
        return s
    mask, depth = _masks(case, gen)
    s |= dict(q=normal(B, T, Hq, D), mask=mask.contiguous(), position=(length[:, None] + depth).to(torch.int32).contiguous(),
              out=torch.zeros(B, T, Hq, D, dtype=dtype, device="cuda"), lse=torch.zeros(B, T, Hq, device="cuda"))
    if own:
        import ancestral_draft_sampling_gb300 as dspark
        s["workspace"] = dspark.TreeWorkspace(B, T, Hq, Hkv, D)
    return s


# ------------------------------------------------------------ the plain forms
def _attend(s):
    c, pool = s["case"], s["pool"][0]
    B, T, Hkv, G, D = c["batch"], c["tokens"], c["kv_heads"], c["group"], c["dim"]
    used = _pages(max(_lengths(c, B)) + T, c["page"])
    kv = pool[:, s["table"][:, :used].long().clamp(min=0)]  # [2, B, pages, heads, page, dim]
    L = used * c["page"]
    kv = kv.transpose(3, 2).reshape(2, B, Hkv, L, D).float()
    q = s["q"].reshape(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D).float()
    scores = (q @ kv[0].transpose(-1, -2)) * (1.0 / math.sqrt(D))
    length, j = s["length"][:, None, None], torch.arange(L, device=q.device)[None, None]
    behind = (j - length).clamp(0, 63)
    sees = (j >= length) & (j < length + T) & (((s["mask"][:, :, None] >> behind) & 1) == 1)
    if s["counts"] is not None:
        sees = sees & (j - length < s["counts"][:, None, None])
    cached = (j < length).expand(B, T, L)
    if c["window"]:
        cached = cached & (s["position"][:, :, None] - j < c["window"])
    sees = (sees | cached)[:, None, :, None].expand(B, 1, T, G, L).reshape(B, 1, T * G, L)
    scores = scores.masked_fill(~sees, -math.inf)
    top = scores.amax(dim=-1, keepdim=True)
    top = torch.where(top == -math.inf, 0.0, top)
    p = (scores - top).exp()
    total = p.sum(dim=-1, keepdim=True)
    out = (p @ kv[1]) / torch.where(total == 0, 1.0, total)
    lse = (top + total.log()).squeeze(-1)

    def rows(x):
        return x.reshape(B, Hkv, T, G, -1).permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, -1)
    out, lse = rows(out).to(s["q"].dtype), rows(lse).squeeze(-1)
    if s["counts"] is not None:  # rows behind the last token stay as they were
        there = (torch.arange(T, device=q.device)[None] < s["counts"][:, None])[..., None]
        out, lse = torch.where(there[..., None], out, s["out"]), torch.where(there, lse, s["lse"])
    return out, lse


def _norm_rotate(x, w, case, cos, sin, eps=1e-6):
    x = x.float()
    if w is not None:
        x = x * (x.square().mean(dim=-1, keepdim=True) + eps).rsqrt() * w
    h = case["rot"] // 2
    r, rest = x[..., :case["rot"]], x[..., case["rot"]:]
    if case["interleaved"]:
        a, b = r[..., 0::2], r[..., 1::2]
        r = torch.stack([a * cos - b * sin, b * cos + a * sin], dim=-1).flatten(-2)
    else:
        a, b = r[..., :h], r[..., h:]
        r = torch.cat([a * cos - b * sin, b * cos + a * sin], dim=-1)
    return torch.cat([r, rest], dim=-1)


def _append(s):
    c = s["case"]
    B, T, h, dtype = c["batch"], c["tokens"], c["rot"] // 2, s["q"].dtype
    angles = s["cos_sin"][s["position"].long()][:, :, None]
    cos, sin = angles[..., :h], angles[..., h:]
    q = _norm_rotate(s["q"], s["wq"], c, cos, sin).to(dtype)
    k = _norm_rotate(s["k"], s["wk"], c, cos, sin).to(dtype)
    t = torch.arange(T, device=q.device)[None]
    there = t < s["counts"][:, None] if s["counts"] is not None else (t >= 0).expand(B, T)
    at = s["length"][:, None] + t
    page = s["table"].gather(1, (at // c["page"]).long()).long()
    b, i = there.nonzero(as_tuple=True)
    pool = s["pool"][0]
    pool[0][page[b, i], :, (at % c["page"])[b, i]] = k[b, i]
    pool[1][page[b, i], :, (at % c["page"])[b, i]] = s["v"][b, i]
    s["q_out"][b, i] = q[b, i]
    return s["q_out"], s["pool"]


def _give(s, ids, order):
    """Takes one hold off each page of ids; those that nobody holds any more
    go back on the free stack, the last of them first."""
    s["ref"].index_add_(0, ids, torch.full_like(ids, -1, dtype=torch.int32))
    first = torch.full_like(s["ref"], 2**31 - 1).scatter_reduce_(0, ids, order, "amin")
    gone = ids[(s["ref"][ids] == 0) & (first[ids] == order)].flip(0)
    n = s["control"][1]
    s["free"][(n + torch.arange(len(gone), device=ids.device)).long()] = gone.to(torch.int32)
    s["control"][1] += len(gone)


def _take(s, wanted):
    """Pages from the top of the free stack for the places of the table that
    `wanted` marks, row by row."""
    rank = wanted.flatten().cumsum(0).reshape(wanted.shape) - 1
    ids = s["free"][(s["control"][1] - 1 - rank).clamp(min=0).long()]
    s["ref"][ids[wanted].long()] = 1
    s["control"][1] -= wanted.sum().to(torch.int32)
    return ids


def _held(s):
    return s["pool"], s["table"], s["count"], s["ref"], s["free"], s["control"][1]


def _accept(s):
    c, table, count, page = s["case"], s["table"], s["count"], s["case"]["page"]
    j = torch.arange(table.shape[1], device=table.device)[None]
    want = (s["length"] + c["tokens"] + page - 1) // page
    more = (j >= count[:, None]) & (j < want[:, None])
    table.copy_(torch.where(more, _take(s, more), table))
    count.copy_(torch.maximum(count, want))
    keep = s["accepted"] + 1
    i = torch.arange(s["path"].shape[1], device=table.device)[None]
    b, i = ((i < keep[:, None]) & (s["path"] != i)).nonzero(as_tuple=True)
    src, dst = s["length"][b] + s["path"][b, i], s["length"][b] + i
    rows = s["pool"][:, :, table[b, (src // page).long()].long(), :, src.long() % page]
    s["pool"][:, :, table[b, dst // page].long(), :, dst % page] = rows
    s["new_length"].copy_(s["length"] + keep)
    left = (s["new_length"] + page - 1) // page
    less = (j >= left[:, None]) & (j < count[:, None])
    _give(s, table[less].long(), torch.arange(table.numel(), device=table.device, dtype=torch.int32).reshape(table.shape)[less])
    table.copy_(torch.where(less, -1, table))
    count.copy_(torch.minimum(count, left))
    return _held(s) + (s["new_length"],)


def _fork(s):
    table, count, page = s["table"], s["count"], s["case"]["page"]
    child, parent = s["child"].long(), s["parent"].long()
    j = torch.arange(table.shape[1], device=table.device)[None]
    old = j < count[child][:, None]
    order = torch.arange(old.numel(), device=table.device, dtype=torch.int32).reshape(old.shape)
    _give(s, table[child][old].long(), order[old])
    full, rest = s["length"] // page, s["length"] % page
    shared, own_page = j < full[:, None], (j == full[:, None]) & (rest > 0)[:, None]
    ids = table[parent]
    s["ref"].index_add_(0, ids[shared].long(), torch.ones_like(ids[shared]))
    table[child] = torch.where(shared, ids, torch.where(own_page, _take(s, own_page), -1))
    count[child] = (full + (rest > 0)).to(torch.int32)
    some = (rest > 0).nonzero().squeeze(1)
    src, dst = ids[some, full[some].long()].long(), table[child[some], full[some].long()].long()
    keep = (torch.arange(page, device=table.device)[None] < rest[some][:, None])[None, None, :, None, :, None]
    s["pool"][:, :, dst] = torch.where(keep, s["pool"][:, :, src], s["pool"][:, :, dst])
    return _held(s)


# ------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if not own:
        if c["op"] == "attend":
            return _attend(s)
        if c["op"] == "append":
            return _append(s)
        return _accept(s) if c["op"] == "accept" else _fork(s)
    import ancestral_draft_sampling_gb300 as dspark
    cache = s["cache"]
    if c["op"] == "attend":
        return dspark.tree_attention(cache, 0, s["q"], s["length"], mask=s["mask"], token_count=s["counts"],
                                     position=s["position"], window=c["window"], out=s["out"], lse=s["lse"],
                                     workspace=s["workspace"])
    if c["op"] == "append":
        dspark.cache_append(cache, 0, s["q"], s["k"], s["v"], s["length"], position=s["position"],
                            cos_sin=s["cos_sin"], q_weight=s["wq"], k_weight=s["wk"], eps=1e-6,
                            interleaved=c["interleaved"], token_count=s["counts"], q_out=s["q_out"])
        return s["q_out"], s["pool"]
    if c["op"] == "accept":
        dspark.cache_reserve(cache, s["length"], c["tokens"])
        dspark.cache_accept(cache, s["length"], s["accepted"], c["tokens"], path=s["path"], new_length=s["new_length"])
        return _held(s) + (s["new_length"],)
    dspark.cache_fork(cache, s["parent"], s["child"], s["length"])
    return _held(s)


def work(case):
    op, page, elt = case["op"], case["page"], ELT[case["dtype"]]
    row = case["kv_heads"] * case["dim"] * elt  # one token's keys or values in one layer
    if op == "fork":
        lens = _lengths(case, case["parents"])
        each = case["children"] // case["parents"]
        copied = sum(n % page for n in lens) * each
        # the copied rows, read once for each parent, and the tables
        tables = sum(_pages(n, page) for n in lens) * (4 + 4 * each)
        return {"bytes": (copied + copied / each) * 2 * case["layers"] * row + tables, "flops": 0}
    lens = _lengths(case, case["batch"])
    if op == "accept":
        moved = sum(_accepted(case))
        return {"bytes": moved * 2 * 2 * case["layers"] * row + 4 * case["batch"] * 12, "flops": 0}
    counts, Hq = _counts(case), case["kv_heads"] * case["group"]
    n = sum(counts)
    if op == "append":
        q = Hq * case["dim"] * elt
        return {"bytes": n * (2 * q + 4 * row + 4 * case["rot"]), "flops": n * (Hq + case["kv_heads"]) * case["dim"] * 10}
    w = case["window"]
    keys = [(min(m, w + case["tokens"] - 1) if w else m) + t for m, t in zip(lens, counts)]
    pairs = sum(k * t for k, t in zip(keys, counts))
    return {"bytes": sum(keys) * 2 * row + n * Hq * (2 * case["dim"] * elt + 4), "flops": 4.0 * pairs * Hq * case["dim"]}


# ------------------------------------------------------------ 64 bits
def exact(case, seed):
    """From the definitions, token by token or request by request, in 64
    bits.  Copies (accept, fork) are no computed numbers."""
    if case["op"] not in ("attend", "append"):
        return None
    s = prepare(case, seed)
    B, T, page, D = case["batch"], case["tokens"], case["page"], case["dim"]
    lens, counts = _lengths(case, B), _counts(case)
    G = case["group"]
    pool = s["pool"][0]
    if case["op"] == "append":
        q_out, kept = s["q_out"].double(), s["pool"].double()
        half = case["rot"] // 2
        at = torch.arange(half, device="cuda")
        first, second = (2 * at, 2 * at + 1) if case["interleaved"] else (at, at + half)
        for b in range(B):
            n = counts[b]
            place = torch.arange(lens[b], lens[b] + n, device="cuda")
            angle = s["cos_sin"][s["position"][b, :n].long()].double()[:, None]
            cos, sin = angle[..., :half], angle[..., half:]
            made = []
            for x, w in ((s["q"][b, :n], s["wq"]), (s["k"][b, :n], s["wk"])):
                x = x.double()
                if w is not None:
                    x = w.double() * x / torch.sqrt((x * x).sum(dim=-1, keepdim=True) / D + 1e-6)
                y = x.clone()
                y[..., first] = x[..., first] * cos - x[..., second] * sin
                y[..., second] = x[..., first] * sin + x[..., second] * cos
                made.append(y)
            q_out[b, :n] = made[0]
            ids = s["table"][b].long()[place // page]
            kept[0, 0, ids, :, place % page] = made[1]
            kept[0, 1, ids, :, place % page] = s["v"][b, :n].double()
        return q_out, kept
    out, lse = s["out"].double(), s["lse"].double()
    for b in range(B):
        n, m = counts[b], lens[b] + counts[b]
        place = torch.arange(m, device="cuda")
        ids = s["table"][b].long()[place // page]
        k, v = (x[ids, :, place % page].double().transpose(0, 1) for x in (pool[0], pool[1]))  # [heads, m, dim]
        bits = torch.stack([(s["mask"][b, :n] >> t) & 1 for t in range(n)], dim=1).bool()
        old = torch.ones(n, lens[b], dtype=torch.bool, device="cuda")
        if case["window"]:
            old = s["position"][b, :n, None] - place[None, :lens[b]] < case["window"]
        sees = torch.cat([old, bits], dim=1)
        for g in range(G):
            heads = torch.arange(case["kv_heads"], device="cuda") * G + g
            z = torch.einsum("thd,hmd->htm", s["q"][b, :n][:, heads].double(), k) / math.sqrt(D)
            z = torch.where(sees[None], z, -math.inf)
            l = torch.logsumexp(z, dim=-1)
            p = torch.where(sees[None], torch.exp(z - torch.where(l == -math.inf, 0.0, l)[..., None]), 0.0)
            out[b, :n, heads] = torch.einsum("htm,hmd->thd", p, v)
            lse[b, :n, heads] = l.transpose(0, 1)
    return out, lse
