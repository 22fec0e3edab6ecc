"""Plain restatement of the paged cache: bounds, block choice, attention over
dequantised rows (float64) and the page tables, taken one sequence after
another.  The formulas are those stated for the paged entry points in
include/hyq.h; the quantiser is ``oracle.quant``."""
from __future__ import annotations

import math

import numpy as np

from .quant import dequantize, quantize

ROWS = 64
EXP_MIN = -40


def step_exponent(amax: float) -> int:
    """Smallest integer e >= EXP_MIN with amax <= 127 * 2^e."""
    e = EXP_MIN
    while 127.0 * 2.0 ** e < amax:
        e += 1
    return e


def bounds(rows):
    """(lo, hi, e) of key rows [n, 128], n >= 1."""
    rows = np.asarray(rows, np.float64)
    e = step_exponent(float(np.abs(rows).max()))
    return (np.floor(rows.min(0) * 2.0 ** -e).astype(np.int64), np.ceil(rows.max(0) * 2.0 ** -e).astype(np.int64), e)


def query_codes(q):
    """Codes of the queries [g, 128] of one KV head's group."""
    q = np.asarray(q, np.float64)
    return np.rint(q * 2.0 ** -step_exponent(float(np.abs(q).max()))).astype(np.int64)


def block_score(codes, lo, hi, e) -> float:
    return float(np.maximum(codes * lo, codes * hi).sum()) * 2.0 ** e


def choose_blocks(scores, k, n_first, n_last):
    """min(n, k) of the n scored blocks, ascending: the first n_first and the
    last n_last, then the largest scores, ties to the lower block."""
    n = len(scores)
    if n <= k:
        return list(range(n))
    forced = [j for j in range(n) if j < n_first or j >= n - n_last]
    rest = sorted((j for j in range(n) if j not in set(forced)), key=lambda j: (-scores[j], j))
    return sorted(forced + rest[:k - len(forced)])


def attend(q, k, v, vis):
    """softmax(q k^T / sqrt(128)) v over the rows ``vis`` (boolean) for one
    query row, and zeros when there is none."""
    if not np.any(vis):
        return np.zeros(q.shape[-1])
    x = (k[vis] @ q) / math.sqrt(q.shape[-1])
    p = np.exp(x - x.max())
    return (p @ v[vis]) / p.sum()


def attend_error(q, k, kparts, vparts, vcodes, vis, out):
    """Elementwise bound of |gpu - attend| for one query row.  kparts, vparts:
    |c s| + |z| of the rows' elements, the sizes of the two products that make a
    dequantised element; vcodes: the values' codes c.

    Value product: a probability p (the largest is 1) is rounded to fp16, and
    p s again, each by half a step: 2^-11 relative, so together 2^-10 of
    sum p (|c s| + |z|); below the normal range of fp16 half a step is 2^-25
    absolute: of p, which meets |c s| + |z|, and of p s, which meets c.  A logit is a
    float32 sum of products with sizes sum |q| (|c s| + |z|), some 20 additions
    deep on the tensor cores, whose additions may truncate: an error below 2^-18
    of that size, in the numerator and in the denominator.  The output is
    rounded to BF16 (2^-8)."""
    if not np.any(vis):
        return np.zeros_like(out)
    x = (k[vis] @ q) / math.sqrt(q.shape[-1])
    p = np.exp(x - x.max())
    size = ((kparts[vis] @ np.abs(q)) / math.sqrt(q.shape[-1])).max()
    mean, total = (p @ vparts[vis]) / p.sum(), (vparts[vis] + vcodes[vis]).sum(0) / p.sum()
    return 2.0 ** -8 * np.abs(out) + mean * (2.0 ** -10 + 2 * 2.0 ** -18 * size) + 2.0 ** -25 * total


def attend_bound(q, k, kparts, vparts, vcodes, vsteps, vis, out):
    """attend_error without a part that does not shrink with the values: the
    kernel keeps probabilities and their products with the value steps at the
    upper end of fp16.

    A row's largest probability is held as at least 2^lift, and every step s
    is taken times 2^F, F >= 0, where
      lift = top - 6, at least 0, with
      top = 15, less 1 for each power of two that the largest step reaches from 1 on;
      2^-F <= 2 max s, or 2^-15 when that is smaller, and F = 0 from max s = 1/2 on.
    Below the normal range of fp16 half a step is 2^-25: of a probability
    2^(-25 - lift), which meets |c s| + |z|, of a product 2^(-25 - lift - F), which
    meets c.  vsteps: the steps of all of the sequence's rows (those of rows that a
    token does not see may count)."""
    if not np.any(vis):
        return np.zeros_like(out)
    x = (k[vis] @ q) / math.sqrt(q.shape[-1])
    p = np.exp(x - x.max())
    size = ((kparts[vis] @ np.abs(q)) / math.sqrt(q.shape[-1])).max()
    most = float(np.asarray(vsteps, np.float64).max())
    top = 15 - (max(0, math.floor(math.log2(most)) + 1) if most > 0 else 0)
    low = 2.0 ** (-25 - max(0, top - 6))
    f = min(1.0, max(2 * most, 2.0 ** -15))
    mean, parts, codes = (p @ vparts[vis]) / p.sum(), vparts[vis].sum(0) / p.sum(), vcodes[vis].sum(0) / p.sum()
    return 2.0 ** -8 * np.abs(out) + mean * (2.0 ** -10 + 2 * 2.0 ** -18 * size) + low * (parts + f * codes)


def dequantised(rows, bits):
    """Rows as the cache holds them, |c s| + |z| of each element, and the codes."""
    c, s, z = quantize(rows, bits)
    val = dequantize(c, s, z)
    zz = np.repeat(z.astype(np.float64), 32, axis=-1)
    return val, np.abs(val - zz) + np.abs(zz), c.astype(np.float64)


class Tables:
    """Page tables with the rules of hyq_pages_*, one sequence after another."""

    def __init__(self, n_pages, n_seqs, max_blocks):
        self.n_pages, self.max_blocks = n_pages, max_blocks
        self.pages = [[] for _ in range(n_seqs)]
        self.lens = [0] * n_seqs

    def refs(self):
        r = [0] * self.n_pages
        for row in self.pages:
            for p in row:
                r[p] += 1
        return r

    def reserve(self, seqs, n_new):
        """The copies (from, to, tiles) of the call, or None when it fails."""
        ok = (len(set(seqs)) == len(seqs) and all(0 <= s < len(self.lens) for s in seqs) and all(n >= 0 for n in n_new))
        if not ok:
            return None
        refs = self.refs()
        want = 0
        for s, n in zip(seqs, n_new):
            blocks = -(-(self.lens[s] + n) // ROWS)
            if blocks > self.max_blocks:
                return None
        free = iter([p for p in range(self.n_pages) if refs[p] == 0])
        rows, lens, copies = [list(r) for r in self.pages], list(self.lens), []
        try:
            for s, n in zip(seqs, n_new):
                if n and lens[s] % ROWS and refs[rows[s][-1]] > 1:
                    old, new = rows[s][-1], next(free)
                    refs[old] -= 1
                    rows[s][-1] = new
                    copies.append((old, new, -(-(lens[s] % ROWS) // 16)))
                want = -(-(lens[s] + n) // ROWS) - len(rows[s])
                rows[s] += [next(free) for _ in range(want)]
                lens[s] += n
        except StopIteration:
            return None
        self.pages, self.lens = rows, lens
        return copies

    def fork(self, src, dst):
        """Pairs left out."""
        bad = []
        todo = []
        for i, (s, d) in enumerate(zip(src, dst)):
            n = len(self.lens)
            if not (0 <= s < n and 0 <= d < n) or d in dst[:i] or d in src or self.lens[d]:
                bad.append(i)
            else:
                todo.append((s, d))
        for s, d in todo:
            self.pages[d], self.lens[d] = list(self.pages[s]), self.lens[s]
        return bad

    def truncate(self, seqs, new_lens):
        bad = []
        for i, (s, n) in enumerate(zip(seqs, new_lens)):
            if not 0 <= s < len(self.lens) or s in seqs[:i] or not 0 <= n <= self.lens[s]:
                bad.append(i)
                continue
            self.lens[s] = n
            self.pages[s] = self.pages[s][:-(-n // ROWS)]
        return bad

    def compact(self):
        """The moves (from, to)."""
        refs = self.refs()
        n = sum(r > 0 for r in refs)
        high = [p for p in range(n, self.n_pages) if refs[p]]
        gaps = [p for p in range(n) if not refs[p]]
        to = dict(zip(high, gaps))
        self.pages = [[to.get(p, p) for p in row] for row in self.pages]
        return list(zip(high, gaps))
