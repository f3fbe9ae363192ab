"""A plain model of the paged cache and of its attention, for the tests: lists
and dictionaries for the bookkeeping, fp64 for the arithmetic.  Shares nothing
with the library."""
import numpy as np


class CacheModel:
    """What exl3_kv_* documents, sequence after sequence and page after page.
    Keys and values are arrays (layers, pages, heads, page_size, dim)."""

    def __init__(self, layers, pages, heads, page_size, dim, seqs, max_pages):
        self.ps, self.max_pages = page_size, max_pages
        self.k = np.zeros((layers, pages, heads, page_size, dim), np.float16)
        self.v = np.zeros_like(self.k)
        self.table = [[] for _ in range(seqs)]
        self.lens = [0] * seqs
        self.refs = [0] * pages

    def pages(self, tokens):
        return -(-tokens // self.ps)

    def extend(self, seqs, counts):
        """False, and nothing changed, where pages or table entries do not suffice."""
        free = [p for p, r in enumerate(self.refs) if r == 0]
        plan = []
        for s, c in zip(seqs, counts):
            n = self.lens[s]
            if self.pages(n + c) > self.max_pages:
                return False
            copy = c > 0 and n % self.ps != 0 and self.refs[self.table[s][-1]] > 1
            plan.append((s, c, copy, self.pages(n + c) - self.pages(n)))
        if sum(copy + fresh for _, _, copy, fresh in plan) > len(free):
            return False
        for s, c, copy, fresh in plan:
            if copy:
                old, new, used = self.table[s][-1], free.pop(0), self.lens[s] % self.ps
                self.k[:, new, :, :used] = self.k[:, old, :, :used]
                self.v[:, new, :, :used] = self.v[:, old, :, :used]
                self.table[s][-1] = new
                self.refs[old] -= 1
                self.refs[new] = 1
            for _ in range(fresh):
                p = free.pop(0)
                self.table[s].append(p)
                self.refs[p] = 1
            self.lens[s] += c
        return True

    def write(self, layer, seqs, counts, k, v):
        for b, (s, c) in enumerate(zip(seqs, counts)):
            for i in range(c):
                pos = self.lens[s] - c + i
                p = self.table[s][pos // self.ps]
                self.k[layer, p, :, pos % self.ps] = k[b, i]
                self.v[layer, p, :, pos % self.ps] = v[b, i]

    def truncate(self, seqs, lens):
        for s, n in zip(seqs, lens):
            n = min(n, self.lens[s])
            while len(self.table[s]) > self.pages(n):
                self.refs[self.table[s].pop()] -= 1
            self.lens[s] = n

    def fork(self, src, dst):
        for a, b in zip(src, dst):
            self.table[b], self.lens[b] = list(self.table[a]), self.lens[a]
            for p in self.table[a]:
                self.refs[p] += 1

    def compact(self):
        n = sum(r > 0 for r in self.refs)
        come = [p for p in range(n, len(self.refs)) if self.refs[p]]
        to = [p for p in range(n) if not self.refs[p]]
        for a, b in zip(come, to):
            self.k[:, b], self.v[:, b] = self.k[:, a], self.v[:, a]
            self.refs[b], self.refs[a] = self.refs[a], 0
        name = dict(zip(come, to))
        self.table = [[name.get(p, p) for p in row] for row in self.table]

    def free_words(self):
        words = np.zeros((len(self.refs) + 31) // 32, np.uint32)
        for p, r in enumerate(self.refs):
            if r == 0:
                words[p // 32] |= np.uint32(1 << (p % 32))
        return words

    def full_table(self, width):
        return np.array([row + [-1] * (width - len(row)) for row in self.table], np.int32)

    def tokens(self, layer, s):
        """Keys and values of a sequence, (tokens, heads, dim) fp64."""
        n = self.lens[s]
        if n == 0:
            z = np.zeros((0,) + (self.k.shape[2], self.k.shape[4]))
            return z, z
        get = lambda a: np.concatenate([a[layer, p] for p in self.table[s]], 1)[:, :n].transpose(1, 0, 2).astype(np.float64)
        return get(self.k), get(self.v)


def visible(pos, n, window, sinks):
    t = np.arange(n)
    see = t <= pos
    if window:
        see &= (t > pos - window) | (t < sinks)
    return see


def attention(q, k, v, first, scale, window=0, sinks=0):
    """Rows q (rows, q_heads, dim) at positions first, first + 1, ... over keys
    and values (tokens, heads, dim), everything fp64.  Returns o, lse and the
    error allowed on each, derived for a kernel that multiplies fp16 operands
    exactly, adds in fp32 and rounds each probability and result to fp16:
      score   a sum of dim products in fp32 (each of its dim/16 + 1 steps off
              by at most 2^-22 of the sum of magnitudes), scaled and taken to
              base 2 (two roundings of 2^-24 each, of the score): d
      p       e^(score) relative: 2 d (its own and the maximum's) + 2^-21, then
              half a step of fp16, 2^-11; it carries a factor of 2^7 or more, so
              below 2^-21 of the largest it is no normal number: half a step of
              2^-24 over that factor, 2^-32 of the largest, absolute
      o       sums of up to n terms in fp32: n/16 + 8 steps of 2^-22 of the sum
              of magnitudes, for o and for the divisor; the result half a step
              of fp16 (2^-11, at least 2^-25 absolute)
    """
    rows, hq, d = q.shape
    n, hk, _ = k.shape
    o, lse = np.zeros((rows, hq, d)), np.full((rows, hq), -np.inf)
    o_tol, lse_tol = np.zeros((rows, hq, d)), np.zeros((rows, hq))
    for i in range(rows):
        see = visible(first + i, n, window, sinks)
        if not see.any():
            continue
        for h in range(hq):
            kk, vv = k[see, h // (hq // hk)], v[see, h // (hq // hk)]
            s = scale * (kk @ q[i, h])
            ds = ((d // 16 + 1) * 2.0 ** -22 * abs(scale) * (np.abs(kk) @ np.abs(q[i, h])) + 2.0 ** -23 * np.abs(s)).max()
            p = np.exp(s - s.max())
            total = p.sum()
            lse[i, h] = s.max() + np.log(total)
            o[i, h] = p @ vv / total
            steps = (len(s) / 16 + 8) * 2.0 ** -22
            mag = p @ np.abs(vv) / total
            o_tol[i, h] = mag * (2.0 ** -11 + 4 * ds + 2 * 2.0 ** -21 + 2 * steps) + \
                2.0 ** -32 * np.abs(vv).sum(0) / total + 2.0 ** -11 * np.abs(o[i, h]) + 2.0 ** -25
            lse_tol[i, h] = 2 * ds + 2.0 ** -21 + steps + 2.0 ** -22 * (1 + abs(lse[i, h]))
    return o, lse, o_tol, lse_tol
