"""The paged cache on the host: page lists, attention of new tokens over them, float64.  TEST
INFRASTRUCTURE ONLY."""
import numpy as np

from ._np import to_np


class Pages:
    """Page tables, lengths and counts under the rules of the library's page management."""

    def __init__(self, table, length, ref, page_size):
        self.table, self.len, self.ref = (np.array(to_np(a), dtype=np.int64) for a in (table, length, ref))
        self.ps = page_size
        self.moves = []          # (source page, destination page, tokens) of the last call
        self.refused = 0

    def _ok(self, row):
        return 0 <= row < len(self.len)

    def extend(self, rows, add):
        free = np.nonzero(self.ref == 0)[0]
        at, seen, self.refused = 0, set(), 0
        for r, n in zip(rows, add):
            new = self.len[r] + n if self._ok(r) else -1
            if not self._ok(r) or r in seen or n < 0 or new > self.table.shape[1] * self.ps:
                self.refused += 1
                seen.add(r)
                continue
            seen.add(r)
            first, last = -(-self.len[r] // self.ps), -(-new // self.ps)
            take = free[at:at + last - first]
            at += last - first
            if len(take) < last - first:
                self.refused += 1
                continue
            self.table[r, first:last] = take
            self.ref[take] = 1
            self.len[r] = new

    def fork(self, parents, children):
        free = np.nonzero(self.ref == 0)[0]
        before, at, seen, self.refused, self.moves = self.len.copy(), 0, set(), 0, []
        for p, c in zip(parents, children):
            if not self._ok(p) or not self._ok(c) or c in seen or before[c] != 0 or p == c:
                self.refused += 1
                seen.add(c)
                continue
            seen.add(c)
            full, part = divmod(int(before[p]), self.ps)
            if part:
                at += 1
                if at > len(free):
                    self.refused += 1
                    continue
                self.table[c, full] = free[at - 1]
                self.ref[free[at - 1]] = 1
                self.moves.append((int(self.table[p, full]), int(free[at - 1]), part))
            self.table[c, :full] = self.table[p, :full]
            np.add.at(self.ref, self.table[p, :full], 1)
            self.len[c] = before[p]

    def free(self, rows):
        seen, self.refused = set(), 0
        for r in rows:
            if not self._ok(r) or r in seen:
                self.refused += 1
                continue
            seen.add(r)
            n = -(-self.len[r] // self.ps)
            np.add.at(self.ref, self.table[r, :n], -1)
            self.table[r, :n] = -1
            self.len[r] = 0

    def compact_into(self, pages):
        """The state of another pool of `pages` pages that the live ones move to."""
        live = np.nonzero(self.ref > 0)[0]
        to = {int(p): i for i, p in enumerate(live)}
        ref = np.zeros(pages, dtype=np.int64)
        ref[:len(live)] = self.ref[live][:pages]
        table = np.array([[to[p] if p >= 0 and to[p] < pages else -1 for p in row] for row in self.table])
        out = Pages(table, self.len, ref, self.ps)
        out.moves = [(p, i, self.ps) for p, i in to.items() if i < pages]
        return out

    def compact(self):
        live = np.nonzero(self.ref > 0)[0]
        holes = [p for p in range(len(live)) if self.ref[p] <= 0]
        movers = [int(p) for p in live if p >= len(live)]
        to = dict(zip(movers, holes))
        self.moves = [(p, h, self.ps) for p, h in to.items()]
        for p, h in to.items():
            self.ref[h], self.ref[p] = self.ref[p], 0
        self.table = np.array([[to.get(int(p), int(p)) for p in row] for row in self.table])


def sequence(pages, table_row, length, layout):
    """[length, Hkv, D] of one sequence, float64."""
    x = to_np(pages)
    ps = x.shape[1] if layout == "NHD" else x.shape[2]
    p = np.asarray(table_row)[:-(-length // ps)]
    y = np.concatenate([x[i] if layout == "NHD" else x[i].swapaxes(0, 1) for i in p]) if len(p) else \
        np.zeros((0, x.shape[2 if layout == "NHD" else 1], x.shape[3]))
    return y[:length]


def attend(q, k, v, scale):
    """Attention of the last len(q) tokens of one sequence, causal: (o, lse, sum p |v|).
    q [n, Hq, D]; k, v [L, Hkv, D]."""
    n, Hq, D = q.shape
    L, Hkv = k.shape[0], k.shape[1]
    g = Hq // Hkv
    o, a = np.zeros((n, Hq, D)), np.zeros((n, Hq, D))
    lse = np.full((n, Hq), -np.inf)
    hidden = np.arange(L)[None] > (L - n + np.arange(n))[:, None]
    some = ~hidden.all(1) if L else np.zeros(n, dtype=bool)
    for h in range(Hq if some.any() else 0):
        s = np.where(hidden, -np.inf, q[:, h] @ k[:, h // g].T * scale)[some]
        m = s.max(1, keepdims=True)
        p = np.exp(s - m)
        lse[some, h] = (m + np.log(p.sum(1, keepdims=True)))[:, 0]
        p /= p.sum(1, keepdims=True)
        o[some, h], a[some, h] = p @ v[:, h // g], p @ np.abs(v[:, h // g])
    return o, lse, a
