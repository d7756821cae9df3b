"""Rotary positions, attention over a paged cache and pages held by several sequences, in 64 bits and plain loops.

The source pages have no counterpart to these operators; "LLM context parallel production guide", section
"位置编码必须跟序列分片一起走", asks that positions follow the shard map, which they do here as data.
"""

from __future__ import annotations

from fractions import Fraction
import math

import numpy as np


def inv_two_pi(bits: int) -> int:
    """floor(2^bits / (2 pi)), pi by Machin's formula 16 arctan(1/5) - 4 arctan(1/239)."""
    n = 2 * bits + 64

    def arctan_inverse(x):
        term = total = (1 << n) // x
        k, sign = 1, -1
        while term:
            term //= x * x
            k += 2
            total += sign * (term // k)
            sign = -sign
        return total

    return (1 << (n + bits)) // (2 * (16 * arctan_inverse(5) - 4 * arctan_inverse(239)))


def rope_turns(inv_freq) -> list:
    """inv_freq / (2 pi) modulo 1 in units of 2^-64, rounded towards zero before the modulus."""
    c = inv_two_pi(400)
    out = []
    for f in inv_freq:
        x = Fraction(float(f)) * c / 2 ** 400
        out.append((1 if x >= 0 else -1) * math.floor(abs(x) * 2 ** 64) % 2 ** 64)
    return out


def rope(x, angle, first=0, adjacent=False, factor=1.0, inverse=False):
    """x [T, heads, d] with pair i of its channels from `first` on, as a complex number, times factor exp(i angle)
    (angle [T, pairs])."""
    out = np.array(x, dtype=np.float64)
    m = angle.shape[1]
    i = np.arange(m)
    re, im = (first + 2 * i, first + 2 * i + 1) if adjacent else (first + i, first + m + i)
    z = (out[..., re] + 1j * out[..., im]) * (factor * np.exp((-1j if inverse else 1j) * angle))[:, None]
    out[..., re], out[..., im] = z.real, z.imag
    return out


def kv_attention(q, k, v, visible, scale):
    """o [n, d_v] and lse [n] of queries q [n, d] over k, v [slots, ...], query t seeing those of visible[t] (an
    index array).  A query that sees none: 0 and -inf."""
    o, lse = np.zeros((len(q), v.shape[1])), np.full(len(q), -np.inf)
    for t, at in enumerate(visible):
        if len(at):
            with np.errstate(invalid="ignore"):  # (inputs that are not finite)
                s = k[at] @ q[t] * scale
                m = s.max()
                e = np.exp(s - m)
                lse[t] = m + np.log(e.sum())
                o[t] = (e / e.sum()) @ v[at]
    return o, lse


class Pages:
    """The pool's counts, and what the calls do to them and to tables (lists of pages)."""

    def __init__(self, refs, page_size):
        self.refs, self.page_size = [int(r) for r in refs], page_size

    def held(self, table, lengths):
        return [[int(p) for p in row[:-(-int(n) // self.page_size)]] for row, n in zip(table, lengths)]

    def counts(self, unmet):
        return [sum(r != 0 for r in self.refs), unmet]

    def _lowest(self):
        return self.refs.index(0) if 0 in self.refs else -1

    def reserve(self, table, lengths, extra):
        rows, unmet = self.held(table, lengths), 0
        for row, n, x in zip(rows, lengths, extra):
            while len(row) > -(-max(int(n) + int(x), 0) // self.page_size):
                self.refs[row.pop()] -= 1
        for row, n, x in zip(rows, lengths, extra):
            while len(row) < -(-(int(n) + int(x)) // self.page_size):
                p = self._lowest()
                unmet += p < 0
                if p >= 0:
                    self.refs[p] = 1
                row.append(p)
        return rows, self.counts(unmet)

    def fork(self, table, lengths, parents):
        """Rows, lengths, counts and the pairs (page, its copy)."""
        rows = self.held(table, lengths)
        for row in rows:
            for p in row:
                self.refs[p] -= 1
        new = [list(rows[p]) if p >= 0 else [] for p in parents]
        n = [int(lengths[p]) if p >= 0 else 0 for p in parents]
        for row, m in zip(new, n):
            for p in row[:m // self.page_size]:
                self.refs[p] += 1
        part = [b for b in range(len(new)) if n[b] % self.page_size]
        kept = []
        for b in part:
            if self.refs[new[b][-1]] == 0:
                self.refs[new[b][-1]] = 1
                kept.append(b)
        pairs, unmet = [], 0
        for b in part:
            if b not in kept:
                p = self._lowest()
                unmet += p < 0
                if p >= 0:
                    self.refs[p] = 1
                    pairs.append((new[b][-1], p))
                new[b][-1] = p
        return new, n, self.counts(unmet), pairs

    def compact(self):
        """Every page's new place (-1: free) and the pairs moved."""
        used = sum(r != 0 for r in self.refs)
        holes = [p for p in range(used) if self.refs[p] == 0]
        movers = [p for p in range(used, len(self.refs)) if self.refs[p] != 0]
        moved = [p if r else -1 for p, r in enumerate(self.refs)]
        for a, b in zip(movers, holes):
            moved[a] = b
            self.refs[b], self.refs[a] = self.refs[a], 0
        return moved, list(zip(movers, holes))
