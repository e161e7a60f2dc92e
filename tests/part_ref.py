"""Plain models of what reads part of the cache, in 64 bits from the
definitions."""
import math

import torch


def page_bounds(keys, page):
    """keys [heads, n, D]: [full pages, heads, 2, D] smallest and largest."""
    out = []
    for i in range(keys.shape[1] // page):
        k = keys[:, i * page:(i + 1) * page]
        out.append(torch.stack([k.amin(dim=1), k.amax(dim=1)], dim=1))
    return torch.stack(out) if out else keys.new_zeros(0, keys.shape[0], 2, keys.shape[2])


def page_scores(q, bounds):
    """q [t, heads, D], bounds [pages, heads_kv, 2, D]: [t, heads_kv, pages] in
    64 bits; what is not a number counts as infinite."""
    t, heads, D = q.shape
    kv = bounds.shape[1]
    g = q.double().reshape(t, kv, heads // kv, 1, D)
    lo, hi = (bounds[:, :, i].double().permute(1, 0, 2)[None, :, None] for i in (0, 1))
    s = torch.maximum(g * lo, g * hi).sum(dim=-1)  # [t, kv, group, pages]
    s = torch.where(torch.isnan(s), math.inf, s)
    return s.amax(dim=2)


def choose(scores, count, first, last):
    """One list: scores of the full pages (64 bits) to ascending page numbers."""
    F = len(scores)
    if F <= count:
        return list(range(F))
    always = set(range(first)) | set(range(F - last, F))
    rest = sorted((j for j in range(F) if j not in always), key=lambda j: (-scores[j], j))
    return sorted(always | set(rest[:count - len(always)]))
