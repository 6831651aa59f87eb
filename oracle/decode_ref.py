"""Plain float64 forms of decoding with drafted tokens over the paged cache: tree
plans and accepted paths, attention of a tree, sampling, compaction, and the pool
of pages.

TEST INFRASTRUCTURE ONLY.  NumPy and plain Python, one element at a time; shares
no code with the HIP path.
"""

from __future__ import annotations

import numpy as np

from .layer_ref import _codes


def tree_parents(parents):
    """One sequence's parents with every value that is no earlier node as -1."""
    return [int(p) if 0 <= int(p) < i else -1 for i, p in enumerate(parents)]


def tree_sees(parents) -> np.ndarray:
    """bool [n][n]: node j is node i or an ancestor of it."""
    up = tree_parents(parents)
    sees = np.zeros((len(up), len(up)), dtype=bool)
    for i in range(len(up)):
        j = i
        while j >= 0:
            sees[i, j] = True
            j = up[j]
    return sees


def tree_accept(parents, draft, sampled):
    """(path, token) of one sequence."""
    up = tree_parents(parents)
    if not up:
        return [], -1
    path = [0]
    while True:
        at = path[-1]
        child = [c for c in range(1, len(up)) if up[c] == at and draft[c] == sampled[at]]
        if not child:
            return path, int(sampled[at])
        path.append(child[0])


def kv_attention_tree(q, cache, table, q_start, kv_len, heads_q: int, sees, sm_scale: float, softcap: float = 0.0):
    """q float64 [tokens][hq d]; sees bool [tokens][>= max_q]: new tokens each node
    sees.  Returns float64 [tokens][hq d], rows of no sequence NaN."""
    k, v, ks, vs = cache["k"], cache["v"], cache["k_scale"], cache["v_scale"]
    pages, heads, page, d = k.shape
    x = np.asarray(q, dtype=np.float64).reshape(len(q), heads_q, d)
    out = np.full(x.shape, np.nan)
    group = heads_q // heads
    for b in range(len(kv_len)):
        n, kv = int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        first = kv - n
        j = np.arange(kv)
        at = np.array([int(table[b][i // page]) for i in j], dtype=np.int64)
        there = (at >= 0) & (at < pages)
        at = np.where(there, at, 0)
        for h in range(heads):
            kh = k[at, h, j % page].astype(np.float64) * ks[at, h].astype(np.float64)[:, None]
            vh = v[at, h, :, j % page].astype(np.float64) * vs[at, h].astype(np.float64)[:, None]
            for i in range(n):
                row = int(q_start[b]) + i
                seen = there & np.array([p < first or bool(sees[row][p - first]) for p in j], dtype=bool)
                for g in range(group):
                    head = h * group + g
                    if not seen.any():
                        out[row, head] = 0.0
                        continue
                    s = kh[seen] @ x[row, head] * sm_scale
                    if softcap:
                        s = softcap * np.tanh(s / softcap)
                    w = np.exp(s - s.max())
                    out[row, head] = w @ vh[seen] / w.sum()
    return out.reshape(len(q), heads_q * d)


def sample(logits, u=0.0, temperature=1.0, top_k=0, top_p=1.0, min_p=0.0):
    """(token, log probability, distance of u from the nearest border as a share of
    the mass) of one row."""
    x = np.asarray(logits, dtype=np.float64)
    x = np.where(np.isnan(x), -np.inf, x)
    if not (x > -np.inf).any():
        return -1, np.nan, 1.0
    order = np.lexsort((np.arange(len(x)), -x))
    if not temperature > 0:
        return int(order[0]), 0.0, 1.0
    y = x[order]
    with np.errstate(invalid="ignore", over="ignore"):
        lw = np.where(y == y[0], 0.0, (y - y[0]) / np.float64(temperature))
    lw = np.where((y == -np.inf) | np.isnan(lw), -np.inf, lw)
    w = np.exp(lw).astype(np.longdouble)
    n = len(w)
    if min_p > 0:
        n = max(1, int((w >= np.longdouble(min(min_p, 1.0))).sum()))
    if 0 < top_k < n:
        n = int(top_k)
    run = np.cumsum(w)
    near = 1.0
    if top_p < 1:
        reach = run[n - 1] * np.longdouble(max(top_p, 0.0))
        near = float(np.min(np.abs(run[:n] - reach)) / run[n - 1]) if n < len(w) or top_p > 0 else 1.0
        n = min(n, int((run[:n] < reach).sum()) + 1)
    u = 0.0 if not u > 0 else min(float(u), 1 - 2.0 ** -48)
    goal = np.longdouble(u) * run[n - 1]
    i = min(int((run[:n] <= goal).sum()), n - 1)
    edges = np.concatenate([[0], run[:n]])
    near = min(near, float(np.min(np.abs(edges - goal)) / run[n - 1]) if u > 0 else 1.0)
    return int(order[i]), float(lw[i] - np.log(run[n - 1])), near


def kv_compact(caches, table, q_start, kv_len, path, count):
    """caches: dicts of NumPy arrays, changed in place; returns the new lengths."""
    out = []
    for b in range(len(kv_len)):
        n, kv = int(q_start[b + 1] - q_start[b]), int(kv_len[b])
        first = kv - n
        if first < 0:
            out.append(kv)
            continue
        nodes = []
        for a in list(path[b])[:max(0, min(int(count[b]), n))]:
            if not (nodes[-1] if nodes else -1) < int(a) < n:
                break
            nodes.append(int(a))
        m = len(nodes)
        out.append(first + m)
        for c in caches:
            pages, heads, page, d = c["k"].shape
            for codes, scale, by_token in ((c["k"], c["k_scale"], True), (c["v"], c["v_scale"], False)):
                for h in range(heads):
                    def token(pos):
                        at = int(table[b][pos // page])
                        if not 0 <= at < pages:
                            return None, np.zeros(d, dtype=np.int8)
                        t = codes[at, h, pos % page] if by_token else codes[at, h, :, pos % page]
                        return scale[at, h], t.copy()

                    def put(pos, t):
                        at = int(table[b][pos // page])
                        if by_token:
                            codes[at, h, pos % page] = t
                        else:
                            codes[at, h, :, pos % page] = t

                    moved = [token(first + a) for a in nodes]
                    for p in range(first // page, (first + m - 1) // page + 1 if m else 0):
                        at = int(table[b][p])
                        here = [i for i in range(m) if (first + i) // page == p]
                        if not 0 <= at < pages or all(nodes[i] == i for i in here):
                            continue
                        kept = [(pos,) + token(pos) for pos in range(p * page, first)]
                        s = max([x[1] for x in kept] + [moved[i][0] for i in here if moved[i][0] is not None],
                                default=np.float32(0))
                        new = [(pos, was, t) for pos, was, t in kept]
                        new += [(first + i,) + moved[i] for i in here]
                        for pos, was, t in new:
                            if was is not None and was != s:
                                t = _codes(t.astype(np.float64) * np.float64(was), s)
                            put(pos, t)
                        scale[at, h] = s
    return out


class Pool:
    """The pool of pages and its page table, changed one row after the other."""

    def __init__(self, pages: int, rows: int, cols: int, page: int):
        self.refs = np.zeros(pages, dtype=np.int64)
        self.table = np.full((rows, cols), -1, dtype=np.int64)
        self.page = page

    def free(self):
        return [p for p in range(len(self.refs)) if self.refs[p] == 0]

    def _valid(self, p):
        return 0 <= p < len(self.refs)

    def resize(self, old, new):
        """Returns (lengths, moved)."""
        rows, cols = self.table.shape
        cut = lambda n: min(max(int(n), 0), cols * self.page)  # noqa: E731
        old, new = [cut(n) for n in old], [cut(n) for n in new]
        pages = lambda n: -(-n // self.page)  # noqa: E731
        for r in range(rows):
            for i in range(pages(new[r]), pages(old[r])):
                p = int(self.table[r, i])
                self.table[r, i] = -1
                if self._valid(p) and self.refs[p] > 0:
                    self.refs[p] -= 1
        lengths, moved, full = [], [], False
        free = self.free()
        for r in range(rows):
            move = (-1, -1)
            have, want = pages(old[r]), pages(new[r])
            if new[r] <= old[r]:
                lengths.append(new[r])
                moved.append(move)
                continue
            last = int(self.table[r, have - 1]) if old[r] % self.page else -1
            copy = self._valid(last) and self.refs[last] > 1
            need = want - have + copy
            full = full or need > len(free)
            if need and full:
                lengths.append(old[r])
                moved.append(move)
                continue
            if copy:
                p = free.pop(0)
                self.refs[last] -= 1
                self.refs[p] = 1
                self.table[r, have - 1] = p
                move = (last, p)
            for i in range(have, want):
                p = free.pop(0)
                self.refs[p] = 1
                self.table[r, i] = p
            lengths.append(new[r])
            moved.append(move)
        return lengths, moved

    def fork(self, src, dst, length):
        for a, b, n in zip(src, dst, length):
            if not (0 <= a < len(self.table) and 0 <= b < len(self.table)) or a == b:
                continue
            for i in range(min(-(-max(int(n), 0) // self.page), self.table.shape[1])):
                p = int(self.table[a, i])
                if self._valid(p) and self.refs[p] > 0:
                    self.refs[p] += 1
                else:
                    p = -1
                self.table[b, i] = p
