"""Paged key-value cache and its attention, in fp64 on the CPU, from the
definitions (one loop per sequence, token and page; nothing shared with the GPU
path).

A cache is an array [pages, page, heads, dim] of the values that it stands for.
"""
from __future__ import annotations

import numpy as np



def visible(position: int, tokens: int, window: int, sinks: int) -> np.ndarray:
    """Which of the tokens 0 .. tokens - 1 a query at `position` sees."""
    t = np.arange(tokens)
    seen = t <= position
    if window:
        seen &= (t > position - window) | (t < sinks)
    return seen


def rows(cache: np.ndarray, table, tokens, head: int) -> np.ndarray:
    """The rows of `tokens` of one sequence and head, [len(tokens), dim]."""
    page = cache.shape[1]
    return np.stack([cache[table[t // page], t % page, head] for t in tokens]).astype(np.float64)


def attend(q, k_cache, v_cache, table, length: int, position: int, head: int, scale: float, window: int, sinks: int):
    """One query row against one kv head.

    Returns (output, lse, bound ingredients): the ingredients are the weighted
    mean of |V| per d, the largest |V| per d, the largest sum_d |q_d K_d| * scale
    of a visible token, and their number.
    """
    tokens = np.flatnonzero(visible(position, max(length, 0), window, sinks))
    dim = len(q)
    if not len(tokens):
        z = np.zeros(dim)
        return z, -np.inf, (z, z, 0.0, 0)
    k, v = rows(k_cache, table, tokens, head), rows(v_cache, table, tokens, head)
    q = np.asarray(q, np.float64)
    with np.errstate(invalid="ignore", over="ignore"):
        s = scale * (k @ q)
        top = s.max()
        w = np.exp(s - top)
        total = w.sum()
        out = (w[:, None] * v).sum(0) / total
        a = (w[:, None] * np.abs(v)).sum(0) / total
        size = scale * (np.abs(k) @ np.abs(q)).max()
        return out, top + np.log(total), (a, np.abs(v).max(0), size, len(tokens))


def e4m3_value(x: np.ndarray) -> np.ndarray:
    """The nearest E4M3 value (ties to even), saturating at +-448; NaN kept."""
    x = np.asarray(x, np.float64)
    with np.errstate(divide="ignore", invalid="ignore"):
        e = np.maximum(np.floor(np.log2(np.abs(x))), -6.0)
        step = np.exp2(np.where(np.isfinite(e), e, -6.0) - 3.0)
        y = np.clip(np.rint(x / step) * step, -448.0, 448.0)
    return np.where(np.isnan(x), np.nan, y)


def append(cache: np.ndarray, new: np.ndarray, tables, lens, cu, scale=None) -> None:
    """Store the rows cu[s] .. cu[s + 1] - 1 of `new` at the end of sequence s."""
    page, pages = cache.shape[1], cache.shape[0]
    for s in range(len(lens)):
        count = cu[s + 1] - cu[s]
        for i in range(count):
            p = int(lens[s]) - count + i
            if p < 0 or p // page >= tables.shape[1] or not 0 <= tables[s, p // page] < pages:
                continue
            x = new[cu[s] + i].astype(np.float64)
            if scale is not None:
                # the quotient is rounded to fp32 before it is rounded to E4M3
                x = e4m3_value((new[cu[s] + i].astype(np.float32) / scale.astype(np.float32)[:, None]).astype(np.float64))
            cache[tables[s, p // page], p % page] = x


class Pages:
    """The page bookkeeping on plain lists; `data` is any array [..., pages, x]."""

    def __init__(self, tables, lens, refs, page: int, data=None):
        self.tables, self.lens, self.refs = np.array(tables), np.array(lens), np.array(refs)
        self.page, self.data = page, data
        self.lacking = 0

    def take(self) -> int:
        free = np.flatnonzero(self.refs == 0)
        if not len(free):
            self.lacking += 1
            return -1
        self.refs[free[0]] = 1
        return int(free[0])

    def reserve(self) -> None:
        self.lacking = 0
        for s in range(len(self.lens)):
            need = -(-max(int(self.lens[s]), 0) // self.page)
            held = [j for j in range(min(need, self.tables.shape[1])) if self.tables[s, j] >= 0]
            for j in range(held[-1] + 1 if held else 0, need):
                if j < self.tables.shape[1]:
                    self.tables[s, j] = self.take()
                else:
                    self.lacking += 1

    def fork(self, parents, children) -> None:
        self.lacking = 0
        copies = []
        for p, c in zip(parents, children):
            if not (0 <= p < len(self.lens) and 0 <= c < len(self.lens)) or p == c:
                continue
            full, rest = divmod(max(int(self.lens[p]), 0), self.page)
            row = np.full(self.tables.shape[1], -1)
            for j in range(min(full, len(row))):
                e = self.tables[p, j]
                if 0 <= e < len(self.refs):
                    row[j] = e
                    self.refs[e] += 1
            if rest and full < len(row) and 0 <= self.tables[p, full] < len(self.refs):
                row[full] = self.take()
                if row[full] >= 0:
                    copies.append((self.tables[p, full], row[full]))
            self.tables[c] = row
            self.lens[c] = max(int(self.lens[p]), 0)
        for a, b in copies:
            self.data[..., b, :] = self.data[..., a, :]

    def drop(self, s: int, j: int) -> None:
        e = self.tables[s, j]
        if e >= 0:
            self.tables[s, j] = -1
            if e < len(self.refs):
                self.refs[e] -= 1

    def free(self, ids) -> None:
        for s in ids:
            if 0 <= s < len(self.lens):
                for j in range(self.tables.shape[1]):
                    self.drop(s, j)
                self.lens[s] = 0

    def trim(self, ids, window: int, sinks: int) -> None:
        for s in ids:
            for j in range(self.tables.shape[1]):
                first, last = j * self.page, (j + 1) * self.page - 1
                if first >= sinks and last <= self.lens[s] - window and not first <= self.lens[s] - 1 <= last:
                    self.drop(s, j)

    def compact(self) -> np.ndarray:
        used = np.flatnonzero(self.refs != 0)
        n = len(used)
        remap = np.full(len(self.refs), -1)
        remap[used] = used
        for a, b in zip(used[used >= n], np.flatnonzero(self.refs[:n] == 0)):
            remap[a] = b
            self.data[..., b, :] = self.data[..., a, :]
            self.refs[b], self.refs[a] = self.refs[a], 0
        good = (self.tables >= 0) & (self.tables < len(self.refs))
        self.tables = np.where(good, remap[np.where(good, self.tables, 0)], np.where(self.tables >= 0, -1, self.tables))
        return remap
