"""Attention over the paged key/value cache that does not read every
sequence's whole context, as cases to be timed and compared.

Long contexts: for each page the smallest and largest keys are kept
(``bounds``), a cheap score of these selects pages for each query (``select``),
and the attention reads the selected pages, the partly filled last one and the
drafted tokens (``sparse``).  Several answers to one prompt: the tokens that a
group of sequences shares are read once for all of them (``prefix``).

Where ``own`` is false, ``run`` computes the operators from elementary torch
operations in 32 bits (the scores, whose order decides, in 64); where it is
true, it calls the framework.
"""
import math

import torch

own = False

DTYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
ELT = {"bf16": 2, "f32": 4}


def listed():
    return [
        # A float32 drafter's cache after a step: few sequences have filled a page.
        dict(name="bounds after a step", op="bounds", dtype="f32", batch=88, tokens=8, kv_heads=8, dim=64, page=16,
             longest=500, layers=5, prompts=False),
        # Three prompts have been written in every layer.
        dict(name="bounds of prompts", op="bounds", dtype="bf16", batch=3, tokens=0, kv_heads=8, dim=128, page=64,
             longest=8191, layers=16, prompts=True),
        # The next token of one request with a very long context.  Latency counts.
        dict(name="select one request", op="select", dtype="bf16", batch=1, tokens=1, kv_heads=8, group=4, dim=128,
             page=64, longest=100000, count=64, first=1, last=2, shared=False, ragged=False),
        # The full serving batch, each drafted token for itself.
        dict(name="select full batch", op="select", dtype="bf16", batch=88, tokens=8, kv_heads=8, group=4, dim=128,
             page=64, longest=16000, count=32, first=1, last=1, shared=False, ragged=True),
        # Float32 queries of an odd shape, one choice for a sequence's tokens.
        dict(name="select f32", op="select", dtype="f32", batch=5, tokens=3, kv_heads=3, group=5, dim=72, page=16,
             longest=3001, count=41, first=0, last=0, shared=True, ragged=True),
        # The next token of one request with a very long context.
        dict(name="sparse one request", op="sparse", dtype="bf16", batch=1, tokens=1, kv_heads=8, group=4, dim=128,
             page=64, longest=100000, count=64, shared=False, mask="causal", ragged=False),
        # The full serving batch with seven drafts each, whose choices mostly agree.
        dict(name="sparse full batch", op="sparse", dtype="bf16", batch=88, tokens=8, kv_heads=8, group=4, dim=128,
             page=64, longest=16000, count=32, shared=False, mask="causal", ragged=True),
        # Wide trees of drafts with one choice for each tree.
        dict(name="sparse wide tree", op="sparse", dtype="bf16", batch=8, tokens=61, kv_heads=8, group=8, dim=128,
             page=32, longest=5000, count=64, shared=True, mask="tree", ragged=False),
        # A float32 drafter's block, which sees itself whole.
        dict(name="sparse block f32", op="sparse", dtype="f32", batch=3, tokens=7, kv_heads=2, group=3, dim=64, page=16,
             longest=2777, count=50, shared=False, mask="full", ragged=True),
        # The first tokens of two answers to one prompt.
        dict(name="prefix pair", op="prefix", dtype="bf16", groups=1, members=2, tokens=1, kv_heads=8, group=4, dim=128,
             page=64, longest=1000, suffix=40, mask="causal", ragged=False),
        # Single tokens of a batch behind one system prompt, small heads and pages.
        dict(name="prefix single tokens", op="prefix", dtype="bf16", groups=1, members=88, tokens=1, kv_heads=8, group=8,
             dim=64, page=16, longest=4000, suffix=2100, mask="causal", ragged=True),
        # Sixteen answers to each of four long prompts, with seven drafts each.
        dict(name="prefix many answers", op="prefix", dtype="bf16", groups=4, members=16, tokens=8, kv_heads=8, group=4,
             dim=128, page=64, longest=16000, suffix=500, mask="causal", ragged=False),
    ]


def _spread(rng, low, high):
    """A whole number between low and high, spread over its logarithm."""
    return min(high, max(low, int(round(math.exp(rng.uniform(math.log(low), math.log(high)))))))


def draw(rng):
    op = rng.choice(["bounds", "select", "select", "sparse", "sparse", "sparse", "prefix", "prefix", "prefix"])
    dtype = rng.choice(["bf16", "bf16", "bf16", "f32"])
    dim, page = rng.choice([64, 128, 128, 96]), rng.choice([16, 32, 64, 128])
    kv, group = rng.choice([1, 2, 3, 4, 8]), rng.randint(1, 8)
    elt = ELT[dtype]
    # float32 and heads of other sizes have a quarter of the largest work
    less = 1 if dtype == "bf16" and dim in (64, 128) else 4
    if op == "bounds":
        prompts = rng.random() < 0.5
        layers, batch = rng.randint(1, 16), _spread(rng, 1, 8 if prompts else 88)
        room = 300_000_000 // (batch * layers * kv * dim * elt)  # tokens, within the largest case
        longest = max(1, min(_spread(rng, 16, 8191), room))
        return dict(op=op, dtype=dtype, batch=batch, tokens=_spread(rng, 1, 64), kv_heads=kv, dim=dim, page=page,
                    longest=longest, layers=layers, prompts=prompts)
    if op == "prefix":
        groups, members, tokens = rng.randint(1, 4), _spread(rng, 1, 88), _spread(rng, 1, 61)
        members = max(1, min(members, 88 // groups))
        longest, suffix = _spread(rng, 64, 16000), _spread(rng, 1, 2100)
        most = 64 * 16500 * 8 * 128 // less  # sequences times keys times heads times dim
        rows = most // (groups * members * kv * dim)
        longest, suffix = max(32, min(longest, rows * 3 // 4)), max(1, min(suffix, rows // 4))
        pairs = 64 * 8 * 11000 * 32 // less  # query rows times keys
        tokens = max(1, min(tokens, pairs // (groups * members * kv * group * (longest + suffix))))
        return dict(op=op, dtype=dtype, groups=groups, members=members, tokens=tokens, kv_heads=kv, group=group, dim=dim,
                    page=page, longest=longest, suffix=suffix, mask=rng.choice(["causal", "tree", "full"]),
                    ragged=rng.random() < 0.5)
    batch, tokens = _spread(rng, 1, 88), _spread(rng, 1, 61)
    longest = max(32, min(_spread(rng, 64, 100000), 88 * 16000 * 8 * 128 // (batch * kv * dim * less)))
    shared = rng.random() < 0.4
    count = max(1, min(_spread(rng, 4, 256), longest // page))
    if op == "select":
        longest = max(longest, 6 * page)
        count = max(1, min(count, longest // (3 * page)))
        first, last = rng.randint(0, min(2, count // 2)), rng.randint(0, min(2, count // 2))
        rows = 88 * 8 * 32 * 250 // less  # query rows times pages
        tokens = max(1, min(tokens, rows // (batch * kv * group * (longest // page + 1))))
        return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, kv_heads=kv, group=group, dim=dim, page=page,
                    longest=longest, count=count, first=first, last=last, shared=shared, ragged=rng.random() < 0.5)
    room = 150_000_000 // less  # keys times dims, within the largest case
    batch = max(1, min(batch, room // (kv * count * page * dim)))
    tokens = max(1, min(tokens, 8 * room // (batch * kv * count * page * dim)))
    return dict(op=op, dtype=dtype, batch=batch, tokens=tokens, kv_heads=kv, group=group, dim=dim, page=page,
                longest=longest, count=count, shared=shared, mask=rng.choice(["causal", "tree", "full"]),
                ragged=rng.random() < 0.5)


# ------------------------------------------------------------ the sizes
def _lengths(case, n):
    """Committed lengths: from a quarter of the longest to the longest, one
    sequence without any where the batch is ragged."""
    top = case["longest"]
    got = [top if b == 0 else max(1, int(top * (0.25 + 0.75 * ((b * 0.6180339887498949) % 1.0)))) for b in range(n)]
    if case.get("ragged") and n > 2:
        got[n // 2] = 0
    return got


def _counts(case, n):
    """Drafted tokens of each sequence: all of them, or from one up."""
    T = case["tokens"]
    if not case.get("ragged"):
        return [T] * n
    return [T if b == 0 else 1 + int(T * ((b * 0.6180339887498949) % 1.0)) for b in range(n)]


def _added(case, n):
    """Tokens that a step has added to each sequence."""
    return [1 + (5 * b + 3) % case["tokens"] for b in range(n)]


def _filled(case):
    """Of each sequence, the lengths before and after and the pages filled between."""
    after = _lengths(case, case["batch"])
    if case["prompts"]:
        before = [0] * len(after)
    else:
        before = [max(0, n - m) for n, m in zip(after, _added(case, len(after)))]
    page = case["page"]
    return before, after, [n // page - m // page for m, n in zip(before, after)]


def _choice(case, pages):
    """Pages that a list names, and those that the lists of a sequence's key
    head name together, of so many full ones."""
    n = min(case["count"], pages)
    if case["shared"] or case["tokens"] == 1:
        return n, n
    return n, min(pages, n + n // 4)


def _prefixes(case):
    """Tokens that each group shares, and what its members have of their own."""
    shared = _lengths(dict(longest=case["longest"]), case["groups"])
    n = case["groups"] * case["members"]
    rest = _lengths(dict(longest=case["suffix"], ragged=case["ragged"]), n)
    # a fork shares full pages: the shared part ends with one
    shared = [max(1, m // case["page"]) * case["page"] for m in shared]
    return shared, rest


def _pages(tokens, page):
    return -(-tokens // page)


# ------------------------------------------------------------ the inputs
def _cache(case, tables, num_pages, gen, layers):
    """A pool and tables [sequences][pages], -1 behind the held ones, as
    tensors: what a program's cache consists of."""
    device = "cuda"
    table = tables.to(torch.int32).contiguous()
    held = table >= 0
    ref = torch.zeros(num_pages, dtype=torch.int32, device=device)
    ref.index_add_(0, table[held].long(), torch.ones_like(table[held]))
    rest = (ref == 0).nonzero().squeeze(1).to(torch.int32)
    free = torch.full((num_pages,), -1, dtype=torch.int32, device=device)
    free[:len(rest)] = rest
    control = torch.zeros(64 + 2 * 1024, dtype=torch.int32, device=device)
    control[1] = len(rest)
    pool = torch.empty(layers, 2, num_pages, case["kv_heads"], case["page"], case["dim"], dtype=DTYPES[case["dtype"]],
                       device=device)
    pool.normal_(generator=gen)
    state = dict(case=case, pool=pool, table=table)
    if own:  # the handle that a program keeps: it names the tensors and holds no data
        import ancestral_draft_sampling_gb300 as dspark
        state["cache"] = dspark.PagedCache.from_tensors(pool, table, held.sum(dim=1).to(torch.int32), ref, free, control)
    return state


def _scatter(held, gen):
    """Tables of sequences that hold held[i] pages each, scattered at random,
    and the number of pages in all (three are free)."""
    total = sum(held)
    order = torch.randperm(total + 3, generator=gen, device="cuda")
    starts = torch.tensor([sum(held[:i]) for i in range(len(held))], device="cuda")
    have = torch.tensor(held, device="cuda")
    j = torch.arange(max(held) + 2, device="cuda")[None]
    return torch.where(j < have[:, None], order[(starts[:, None] + j).clamp(max=total + 2)], -1), total + 3


def _bounds_of(keys):
    """Smallest and largest keys of pages [..., slots, dim]."""
    return torch.stack([keys.amin(dim=-2), keys.amax(dim=-2)], dim=-2)


def _masks(case, B, gen):
    """For each drafted token the drafted tokens that it sees (bit j: token j)."""
    T = case["tokens"]
    one = torch.ones(B, T, dtype=torch.int64, device="cuda")
    t = torch.arange(T, device="cuda")
    if case["mask"] == "full":
        return torch.full_like(one, (1 << T) - 1)
    if case["mask"] == "causal":
        return (one << (t + 1)) - 1
    mask = one.clone()
    parents = (torch.rand(B, T, generator=gen, device="cuda") * t).long()
    rows = torch.arange(B, device="cuda")
    for i in range(1, T):
        mask[:, i] = mask[rows, parents[:, i]] | (one[:, i] << i)
    return mask


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op, dtype, page, Hkv, D = case["op"], DTYPES[case["dtype"]], case["page"], case["kv_heads"], case["dim"]
    i32 = dict(dtype=torch.int32, device="cuda")
    if op == "bounds":
        before, after, _ = _filled(case)
        tables, total = _scatter([max(1, _pages(n, page)) for n in after], gen)
        s = _cache(case, tables, total, gen, case["layers"])
        s |= dict(start=torch.tensor(before, **i32), length=torch.tensor(after, **i32),
                  bounds=torch.randn(case["layers"], total, Hkv, 2, D, generator=gen, device="cuda").to(dtype))  # of before
        return s
    T, Hq = case["tokens"], Hkv * case["group"]
    if op == "prefix":
        shared, rest = _prefixes(case)
        M = case["members"]
        B = case["groups"] * M
        lens = [shared[b // M] + rest[b] for b in range(B)]
        own_pages, total = _scatter([_pages(rest[b] + T, page) for b in range(B)] + [n // page for n in shared], gen)
        j = torch.arange(max(_pages(n + T, page) for n in lens) + 2, device="cuda")[None].expand(B, -1)
        full = torch.tensor([shared[b // M] // page for b in range(B)], device="cuda")[:, None]
        at = (j - full).clamp(0, own_pages.shape[1] - 1)
        mine = torch.where(j - full < own_pages.shape[1], own_pages[:B].gather(1, at), -1)
        theirs = own_pages[B:][torch.arange(B, device="cuda") // M].gather(1, j.clamp(max=own_pages.shape[1] - 1))
        s = _cache(case, torch.where(j < full, theirs, mine), total, gen, 1)
        s |= dict(group_start=torch.arange(case["groups"] + 1, **i32) * M, prefix=torch.tensor(shared, **i32))
    else:
        B = case["batch"]
        lens = _lengths(case, B)
        tables, total = _scatter([_pages(n + T, page) for n in lens], gen)
        s = _cache(case, tables, total, gen, 1)
    counts = torch.tensor(_counts(case, B), **i32)
    q = torch.randn(B, T, Hq, D, generator=gen, device="cuda").to(dtype)
    s |= dict(length=torch.tensor(lens, **i32), counts=counts if case["ragged"] else None, q=q)
    if op == "select":
        s["bounds"] = _bounds_of(s["pool"][:, 0])
        s["pages"] = torch.zeros(B, 1 if case["shared"] else T, Hkv, case["count"], **i32)
        if own:
            import ancestral_draft_sampling_gb300 as dspark
            s["workspace"] = dspark.SelectWorkspace(s["cache"], B, T)
        return s
    s |= dict(mask=_masks(case, B, gen).contiguous(), out=torch.zeros(B, T, Hq, D, dtype=dtype, device="cuda"),
              lse=torch.zeros(B, T, Hq, device="cuda"))
    if op == "sparse":
        # Each sequence and key head has pages that its tokens agree upon, of
        # which each token's list leaves out some.
        F = torch.tensor([n // page for n in lens], device="cuda")
        most = max(1, max(lens) // page)
        Ts = 1 if case["shared"] else T
        some = torch.rand(B, 1, Hkv, most, generator=gen, device="cuda")
        some = torch.where(torch.arange(most, device="cuda") < F[:, None, None, None], some, 2.0)
        width = min(most, case["count"] + case["count"] // 4)
        agreed = some.argsort(dim=-1)[..., :width].expand(B, Ts, Hkv, width)
        sizes = torch.tensor([_choice(case, n // page) for n in lens], device="cuda")
        liked = torch.rand(B, Ts, Hkv, width, generator=gen, device="cuda")
        liked = torch.where(torch.arange(width, device="cuda") < sizes[:, 1, None, None, None], liked, 2.0)
        order = liked.argsort(dim=-1)[..., :case["count"]]
        chosen = agreed.gather(-1, order)
        there = torch.arange(chosen.shape[-1], device="cuda") < sizes[:, 0, None, None, None]
        chosen = torch.where(there, chosen, 1 << 40).sort(dim=-1).values
        pages = torch.full((B, Ts, Hkv, case["count"]), -1, **i32)
        pages[..., :chosen.shape[-1]] = torch.where(chosen < 1 << 40, chosen, -1).to(torch.int32)
        s["pages"] = pages
    if own:
        import ancestral_draft_sampling_gb300 as dspark
        if op == "sparse":
            s["workspace"] = dspark.SparseWorkspace(s["cache"], B, T, Hq, case["count"])
        else:
            s["workspace"] = dspark.PrefixWorkspace(B, T, Hq, Hkv, D)
    return s


# ------------------------------------------------------------ the plain forms
def _bounds(s):
    page, table = s["case"]["page"], s["table"]
    ends = (torch.arange(table.shape[1], device=table.device)[None] + 1) * page
    ids = table[(ends > s["start"][:, None]) & (ends <= s["length"][:, None])].long()
    s["bounds"][:, ids] = _bounds_of(s["pool"][:, 0, ids])
    return s["bounds"]


def _select(s):
    c = s["case"]
    B, T, Hkv, G, D, P = c["batch"], c["tokens"], c["kv_heads"], c["group"], c["dim"], c["count"]
    most = max(1, max(_lengths(c, B)) // c["page"])
    edge = s["bounds"][0][s["table"][:, :most].long().clamp(min=0)].double()  # [B, pages, heads, 2, dim]
    edge = edge.permute(0, 2, 3, 4, 1)  # [B, heads, 2, dim, pages]
    q = s["q"].double().reshape(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    score = q.clamp(max=0.0) @ edge[:, :, 0] + q.clamp(min=0.0) @ edge[:, :, 1]
    score = score.reshape(B, Hkv, T, G, most).amax(dim=3).transpose(1, 2)  # [B, T, heads, pages]
    there = torch.ones(B, T, dtype=torch.bool, device=q.device)
    if s["counts"] is not None:
        there = torch.arange(T, device=q.device)[None] < s["counts"][:, None]
    if c["shared"]:
        score = torch.where(there[:, :, None, None], score, -math.inf).amax(dim=1, keepdim=True)
        there = there[:, :1]
    j = torch.arange(most, device=q.device)
    F = (s["length"] // c["page"])[:, None, None, None]
    score = torch.where((j < c["first"]) | (j >= F - c["last"]), math.inf, score)
    score = torch.where(j < F, score, -math.inf)
    order = score.sort(dim=-1, descending=True, stable=True).indices[..., :P]
    order = torch.where(torch.arange(order.shape[-1], device=q.device) < F, order, 1 << 40).sort(dim=-1).values
    got = torch.full_like(s["pages"], -1)
    got[..., :order.shape[-1]] = torch.where(order < 1 << 40, order, -1).to(torch.int32)
    s["pages"].copy_(torch.where(there[:, :, None, None], got, s["pages"]))
    return s["pages"]


def _softmax(scores, values):
    """Several parts' scores [..., rows, keys] (-inf: hidden) and values [..., keys,
    dim]: the weighted values and the log-sum-exp."""
    top = scores[0].amax(dim=-1, keepdim=True)
    for x in scores[1:]:
        top = torch.maximum(top, x.amax(dim=-1, keepdim=True))
    top = torch.where(top == -math.inf, 0.0, top)
    total, out = 0.0, 0.0
    for x, v in zip(scores, values):
        p = (x - top).exp()
        total = total + p.sum(dim=-1, keepdim=True)
        out = out + p @ v
    return out / torch.where(total == 0, 1.0, total), (top + total.log()).squeeze(-1)


def _behind(s, at, B, T):
    """Which of the places at [B, keys] behind the committed tokens each
    token sees: [B, T, keys]."""
    j = at - s["length"][:, None]
    sees = ((j >= 0) & (j < T))[:, None] & (((s["mask"][:, :, None] >> j.clamp(0, 63)[:, None]) & 1) == 1)
    if s["counts"] is not None:
        sees = sees & (j < s["counts"][:, None])[:, None]
    return sees


def _written(s, out, lse):
    """Rows behind the last token of a sequence stay as they were."""
    out = out.to(s["q"].dtype)
    if s["counts"] is not None:
        there = (torch.arange(out.shape[1], device=out.device)[None] < s["counts"][:, None])[..., None]
        out, lse = torch.where(there[..., None], out, s["out"]), torch.where(there, lse, s["lse"])
    return out, lse


def _sparse(s):
    c, (pk, pv), page = s["case"], s["pool"][0], s["case"]["page"]
    B, T, Hkv, G, D, P = c["batch"], c["tokens"], c["kv_heads"], c["group"], c["dim"], c["count"]
    Ts = s["pages"].shape[1]
    rows = T * G // Ts  # rows of a list
    q = s["q"].float().reshape(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, Ts, rows, D)
    pages = s["pages"].permute(0, 2, 1, 3).long()  # [B, heads, lists, P]
    ids = s["table"].long()[torch.arange(B, device=q.device)[:, None, None, None], pages.clamp(min=0)]
    heads = torch.arange(Hkv, device=q.device)[None, :, None, None]
    k, v = (x[ids, heads].float().reshape(B, Hkv, Ts, P * page, D) for x in (pk, pv))
    scale = 1.0 / math.sqrt(D)
    one = (q @ k.transpose(-1, -2)) * scale
    one = one.masked_fill((pages < 0).repeat_interleave(page, dim=-1)[..., None, :], -math.inf)
    # the tokens behind the full pages
    at = (s["length"] // page * page)[:, None] + torch.arange(page + T, device=q.device)[None]
    ids = s["table"].gather(1, (at // page).clamp(max=s["table"].shape[1] - 1)).long().clamp(min=0)
    k2, v2 = (x[ids, :, at % page].float().permute(0, 2, 1, 3)[:, :, None] for x in (pk, pv))  # [B, heads, 1, keys, dim]
    sees = (at < s["length"][:, None])[:, None] | _behind(s, at, B, T)
    sees = sees[:, :, None].expand(-1, -1, G, -1).reshape(B, 1, Ts, rows, -1)
    two = ((q @ k2.transpose(-1, -2)) * scale).masked_fill(~sees, -math.inf)
    out, lse = _softmax([one, two], [v, v2])
    out = out.reshape(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, D)
    return _written(s, out, lse.reshape(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hkv * G))


def _prefix(s):
    c, (pk, pv), page = s["case"], s["pool"][0], s["case"]["page"]
    M, T, Hkv, G, D = c["members"], c["tokens"], c["kv_heads"], c["group"], c["dim"]
    B = c["groups"] * M
    shared, rest = _prefixes(c)
    q = s["q"].float().reshape(B, T, Hkv, G, D).permute(0, 2, 1, 3, 4).reshape(B, Hkv, T * G, D)
    scale = 1.0 / math.sqrt(D)
    start = s["prefix"].long().repeat_interleave(M)[:, None]
    at = start + torch.arange(max(rest) + T, device=q.device)[None]
    ids = s["table"].gather(1, (at // page).clamp(max=s["table"].shape[1] - 1)).long().clamp(min=0)
    k2, v2 = (x[ids, :, at % page].float().permute(0, 2, 1, 3) for x in (pk, pv))  # [B, heads, keys, dim]
    sees = (at < s["length"][:, None])[:, None] | _behind(s, at, B, T)
    sees = sees[:, :, None].expand(-1, -1, G, -1).reshape(B, 1, T * G, -1)
    two = ((q @ k2.transpose(-1, -2)) * scale).masked_fill(~sees, -math.inf)
    outs, lses = [], []
    for g in range(c["groups"]):  # the shared keys once for all rows of a group
        m = slice(g * M, (g + 1) * M)
        ids = s["table"][g * M, :shared[g] // page].long()
        k, v = (x[ids].float().transpose(0, 1).reshape(Hkv, shared[g], D) for x in (pk, pv))
        one = (q[m] @ k.transpose(-1, -2)) * scale
        out, lse = _softmax([one, two[m]], [v, v2[m]])
        outs.append(out)
        lses.append(lse)
    out = torch.cat(outs).reshape(B, Hkv, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hkv * G, D)
    return _written(s, out, torch.cat(lses).reshape(B, Hkv, T, G).permute(0, 2, 1, 3).reshape(B, T, Hkv * G))


# ------------------------------------------------------------ one pass
def run(s):
    c = s["case"]
    if not own:
        return {"bounds": _bounds, "select": _select, "sparse": _sparse, "prefix": _prefix}[c["op"]](s)
    import ancestral_draft_sampling_gb300 as dspark
    cache = s["cache"]
    if c["op"] == "bounds":
        return dspark.cache_bounds(cache, s["start"], s["length"], bounds=s["bounds"])
    if c["op"] == "select":
        return dspark.select_pages(cache, 0, s["bounds"], s["q"], s["length"], c["count"], first=c["first"],
                                   last=c["last"], shared=c["shared"], token_count=s["counts"], pages=s["pages"],
                                   workspace=s["workspace"])
    if c["op"] == "sparse":
        return dspark.sparse_attention(cache, 0, s["q"], s["length"], s["pages"], mask=s["mask"],
                                       token_count=s["counts"], out=s["out"], lse=s["lse"], workspace=s["workspace"])
    return dspark.prefix_attention(cache, 0, s["q"], s["length"], s["group_start"], s["prefix"], mask=s["mask"],
                                   token_count=s["counts"], out=s["out"], lse=s["lse"], workspace=s["workspace"])


def work(case):
    op, page, elt, D, Hkv = case["op"], case["page"], ELT[case["dtype"]], case["dim"], case["kv_heads"]
    row = Hkv * D * elt  # one token's keys or values in one layer
    if op == "bounds":
        filled = sum(_filled(case)[2])
        return {"bytes": filled * case["layers"] * (page + 2) * row + 8 * case["batch"],
                "flops": 2 * filled * case["layers"] * page * Hkv * D}
    T, Hq = case["tokens"], Hkv * case["group"]
    if op == "prefix":
        shared, rest = _prefixes(case)
        M = case["members"]
        B = case["groups"] * M
        counts = _counts(case, B)
        keys = sum(shared) + sum(r + t for r, t in zip(rest, counts))
        pairs = sum((shared[b // M] + rest[b] + counts[b]) * counts[b] for b in range(B))
        return {"bytes": keys * 2 * row + sum(counts) * Hq * (2 * D * elt + 4), "flops": 4.0 * pairs * Hq * D}
    B = case["batch"]
    lens, counts = _lengths(case, B), _counts(case, B)
    n = sum(counts)
    if op == "select":
        pages = [m // page for m in lens]
        lists = B if case["shared"] else n
        return {"bytes": sum(pages) * 2 * row + n * Hq * D * elt + lists * Hkv * case["count"] * 4,
                "flops": 4.0 * sum(p * t for p, t in zip(pages, counts)) * Hq * D}
    keys = pairs = lists = 0
    for m, t in zip(lens, counts):
        listed_pages, together = _choice(case, m // page)
        if t == 1:
            together = listed_pages
        keys += together * page + m % page + t
        pairs += (listed_pages * page + m % page + t) * t
        lists += listed_pages * (1 if case["shared"] else t)
    return {"bytes": keys * 2 * row + n * Hq * (2 * D * elt + 4) + lists * Hkv * 4, "flops": 4.0 * pairs * Hq * D}


# ------------------------------------------------------------ 64 bits
def _attend(q, k, v, sees):
    """One sequence: q [tokens, heads, group, dim], k and v [heads, (tokens,)
    keys, dim], sees [tokens, keys] or [heads, tokens, keys]."""
    if sees.dim() == 2:
        sees = sees[None]
    if k.dim() == 3:
        z = torch.einsum("thgd,hmd->htgm", q, k)
    else:
        z = torch.einsum("thgd,htmd->htgm", q, k)
    z = torch.where(sees[:, :, None], z / math.sqrt(q.shape[-1]), -math.inf)
    l = torch.logsumexp(z, dim=-1)
    p = torch.where(z == -math.inf, 0.0, torch.exp(z - torch.where(l == -math.inf, 0.0, l)[..., None]))
    o = torch.einsum("htgm,hmd->thgd" if v.dim() == 3 else "htgm,htmd->thgd", p, v)
    return o, l.permute(1, 0, 2)


def exact(case, seed):
    """From the definitions, sequence by sequence, in 64 bits.  Chosen pages
    are whole numbers."""
    op, page, Hkv, D = case["op"], case["page"], case["kv_heads"], case["dim"]
    if op == "select":
        return None
    s = prepare(case, seed)
    if op == "bounds":
        got = s["bounds"].double()
        before, after, _ = _filled(case)
        for b, (m, n) in enumerate(zip(before, after)):
            for i in range(m // page, n // page):
                p = int(s["table"][b, i])
                keys = s["pool"][:, 0, p].double()
                got[:, p, :, 0], got[:, p, :, 1] = keys.min(dim=2).values, keys.max(dim=2).values
        return got
    T, G, pool = case["tokens"], case["group"], s["pool"][0]
    out, lse = s["out"].double(), s["lse"].double()
    B = out.shape[0]
    lens, counts = s["length"].tolist(), _counts(case, B)
    for b in range(B):
        n, m = counts[b], lens[b]
        q = s["q"][b, :n].double().reshape(n, Hkv, G, D)
        drafted = torch.stack([(s["mask"][b, :n] >> t) & 1 for t in range(n)], dim=1).bool()
        ids = s["table"][b].long()
        if op == "prefix":
            place = torch.arange(m + n, device="cuda")
            k, v = (x[ids[place // page], :, place % page].double().transpose(0, 1) for x in (pool[0], pool[1]))
            sees = torch.cat([torch.ones(n, m, dtype=torch.bool, device="cuda"), drafted], dim=1)
        else:
            place = torch.arange(m // page * page, m + n, device="cuda")
            tail = [x[ids[place // page], :, place % page].double().transpose(0, 1) for x in (pool[0], pool[1])]
            sees = torch.cat([torch.ones(n, m % page, dtype=torch.bool, device="cuda"), drafted], dim=1)
            pages = s["pages"][b].transpose(0, 1).long()  # [heads, lists, P]
            pages = pages[:, :n] if pages.shape[1] > 1 else pages
            heads = torch.arange(Hkv, device="cuda")[:, None, None]
            k, v = (torch.cat([x[ids[pages.clamp(min=0)], heads].double().flatten(2, 3),
                               y[:, None].expand(-1, pages.shape[1], -1, -1)], dim=2)
                    for x, y in zip((pool[0], pool[1]), tail))
            listed_too = (pages >= 0).repeat_interleave(page, dim=-1)
            sees = torch.cat([listed_too.expand(-1, n, -1), sees[None].expand(Hkv, -1, -1)], dim=2)
            if pages.shape[1] == 1:
                k, v = k[:, 0], v[:, 0]
        o, l = _attend(q, k, v, sees)
        out[b, :n], lse[b, :n] = o.reshape(n, Hkv * G, D), l.reshape(n, Hkv * G)
    return out, lse
