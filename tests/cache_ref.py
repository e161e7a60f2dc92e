"""Plain models of the paged cache and the attention over it: the bookkeeping
as Python lists, the numerics in 64 bits from the definitions."""
import math

import numpy as np
import torch


class PageModel:
    """What the bookkeeping calls do, one entry at a time."""

    def __init__(self, num_pages, page, max_seqs, max_pages):
        self.page, self.max_pages = page, max_pages
        self.held = [[] for _ in range(max_seqs)]
        self.free = list(range(num_pages))[::-1]
        self.ref = [0] * num_pages
        self.error = 0

    def reserve(self, seq, length, tokens):
        need = []
        for s, n in zip(seq, length):
            if not 0 <= s < len(self.held) or n < 0:
                self.error, more = (6 if n >= 0 else 7), 0
                more = 0
            else:
                want = -(-(n + tokens) // self.page)
                more = max(0, want - len(self.held[s]))
                if want > self.max_pages:
                    self.error, more = 8, 0
            need.append(more)
        left = len(self.free)
        for s, more in zip(seq, need):
            if more > left:
                self.error = 8
                continue
            left -= more
            for _ in range(more):
                p = self.free.pop()
                self.ref[p] = 1
                self.held[s].append(p)

    def give(self, entries):
        """entries: (sequence, index) in order; the last goes back first."""
        pages = [self.held[s][i] for s, i in entries]
        for p in pages:
            self.ref[p] -= 1
        gone = []
        for p in pages:
            if self.ref[p] == 0 and p not in gone:
                gone.append(p)
        self.free += gone[::-1]
        for s, i in sorted(entries, reverse=True):
            del self.held[s][i:]

    def release(self, seq):
        self.give([(s, i) for s in seq if 0 <= s < len(self.held) for i in range(len(self.held[s]))])

    def accept(self, seq, length, keep):
        now = [n + k for n, k in zip(length, keep)]
        self.give([(s, i) for s, n in zip(seq, now) if 0 <= s < len(self.held) and n >= 0
                   for i in range(-(-n // self.page), len(self.held[s]))])
        return now

    def fork(self, parent, child, length):
        """Returns the copies to make: (from page, to page, rows)."""
        ok = [0 <= p < len(self.held) and 0 <= c < len(self.held) for p, c in zip(parent, child)]
        kids = [c for c, o in zip(child, ok) if o]
        if len(set(kids)) < len(kids) or set(kids) & set(parent):
            self.error = 11
            return []
        self.release(kids)
        copies, wants = [], []
        for p, c, n, o in zip(parent, child, length, ok):
            if not o:
                self.error = 6
            elif n < 0 or n > len(self.held[p]) * self.page:
                self.error = 7
            else:
                wants.append((p, c, n))
        for p, c, n in wants:
            full, rest = divmod(n, self.page)
            if rest and not self.free:
                self.error = 8
                continue
            self.held[c] = self.held[p][:full]
            for q in self.held[c]:
                self.ref[q] += 1
            if rest:
                q = self.free.pop()
                self.ref[q] = 1
                self.held[c].append(q)
                copies.append((self.held[p][full], q, rest))
        return copies

    def check(self, cache):
        """The cache's tables are this model's."""
        n = int(cache.control[1])
        assert n == len(self.free) and cache.free_list[:n].tolist() == self.free
        assert cache.ref_count.tolist() == self.ref
        assert cache.page_count.tolist() == [len(h) for h in self.held]
        table = cache.block_table.cpu().numpy()
        for row, held in zip(table, self.held):
            assert row[:len(held)].tolist() == held and (row[len(held):] == -1).all()
        assert int(cache.control[2]) == 0


def place(cache, s, n):
    """Pages and slots of the first n tokens of sequence s (on the host)."""
    at = torch.arange(n)
    return cache.block_table[s].cpu().long()[at // cache.page_size], at % cache.page_size


def rotate(x, w, eps, cos_sin, position, interleaved):
    """float64 [.., heads, D]: the normalised and rotated rows, and the sum of
    the magnitudes that each value is made of."""
    x = x.double()
    if w is not None:
        x = x / torch.sqrt((x * x).mean(dim=-1, keepdim=True) + eps) * w.double()
    rot = cos_sin.shape[1]
    h = rot // 2
    at = torch.arange(h)
    i, j = (2 * at, 2 * at + 1) if interleaved else (at, at + h)
    c = cos_sin.double()[position.long()][..., None, :h]
    s = cos_sin.double()[position.long()][..., None, h:]
    y, size = x.clone(), x.abs()
    y[..., i] = x[..., i] * c - x[..., j] * s
    y[..., j] = x[..., j] * c + x[..., i] * s
    size[..., i] = (x[..., i] * c).abs() + (x[..., j] * s).abs()
    size[..., j] = (x[..., j] * c).abs() + (x[..., i] * s).abs()
    return y, size


def attend(k, v, q, sees, scale):
    """One sequence in 64 bits: k, v [heads_kv, n, D], q [t, heads, D], sees
    [t, n].  Returns out, lse, and the parts of the error bound: sum p |v| and
    the largest |q| |k| scale of each row."""
    t, heads, D = q.shape
    group = heads // k.shape[0]
    out, lse = torch.zeros(t, heads, D, dtype=torch.float64), torch.full((t, heads), -math.inf, dtype=torch.float64)
    size, reach = torch.zeros(t, heads, D, dtype=torch.float64), torch.zeros(t, heads, dtype=torch.float64)
    for h in range(heads):
        K, V = k[h // group].double(), v[h // group].double()
        for i in range(t):
            see = sees[i]
            if not see.any():
                continue
            z = (K[see] @ q[i, h].double()) * scale
            m = z.max()
            p = torch.exp(z - m)
            out[i, h] = (p @ V[see]) / p.sum()
            size[i, h] = (p @ V[see].abs()) / p.sum()
            lse[i, h] = m + torch.log(p.sum())
            reach[i, h] = (K[see].abs() @ q[i, h].double().abs()).max() * abs(scale)
    return out, lse, size, reach


def attend_bounds(size, reach, out, lse, n, D, bf16):
    """How far a kernel may be off, from the roundings it makes.

    Scores: D products and sums of float32, |error| <= (D + 8) u |q||k| scale
    with u = 2^-24 (the additions' errors grow with the partial sums, which
    |q||k| bounds); a weight's relative error is that of its score and of the
    maximum's (which cancels in the quotient only up to rounding), 8 u for
    exp and its argument scaled to base 2 (|score| u more, again below
    |q||k| u).  Sums of n terms: n u relative to sum p |v|, numerator and
    denominator.  bfloat16: weights rounded to 2^-8 of themselves, the result
    to 2^-8 of itself."""
    u = 2.0 ** -24
    score = (D + 16) * u * reach
    w = 2 * score + (2 * n + 32) * u
    if bf16:
        w = w + 2.0 ** -8
    bound = size * w[..., None]
    if bf16:
        bound = bound + 2.0 ** -8 * (out.abs() + bound)
    else:
        bound = bound + u * out.abs()
    finite = torch.where(torch.isfinite(lse), lse.abs(), torch.zeros_like(lse))
    return bound, score + (n + 32) * u + 4 * u * finite


def tree_sees(length, count, words, window, position):
    """[count, length + count] which keys each drafted token sees."""
    n = length + count
    sees = torch.zeros(count, n, dtype=torch.bool)
    for t in range(count):
        lo = 0
        if window:
            lo = max(0, max(int(position[t]), length) - window + 1)
        sees[t, min(lo, length):length] = True
        for j in range(count):
            sees[t, length + j] = bool((int(words[t]) >> j) & 1)
    return sees


def tree_words(kind, T, rng):
    """T mask words as Python ints in 0 .. 2^64 - 1, and the depths."""
    if kind == "causal":
        return [(2 << t) - 1 for t in range(T)], list(range(T))
    if kind == "full":
        return [(1 << T) - 1] * T, list(range(T))
    words, depth = [], []
    for t in range(T):
        p = int(rng.integers(0, t)) if t else -1
        words.append((words[p] if t else 0) | (1 << t))
        depth.append(depth[p] + 1 if t else 0)
    if kind == "holes":  # some tokens see nothing of the tree
        words = [0 if rng.random() < 0.4 else w for w in words]
    return words, depth


def as_int64(words):
    return torch.from_numpy(np.array(words, dtype=np.uint64).view(np.int64).copy())
