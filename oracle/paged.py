"""The paged 8-bit cache in 64 bits: a Python model of the slots, the pages and
what they hold, and dense attention over it."""
from __future__ import annotations

import numpy as np

PAGE, DIM, E_MIN, E_MAX, TOP = 64, 256, -40, 60, 448.0
BF16_MAX = float(np.float32(np.uint32(0x7F7F0000).view(np.float32)))


def e4m3(y: np.ndarray) -> np.ndarray:
    """The nearest e4m3 value (ties to the even multiple of the step), saturating."""
    y = np.asarray(y, dtype=np.float64)
    size = np.frexp(np.maximum(np.abs(y), 2.0**-6))[1] - 1  # 2^size <= |y| (or e4m3's least normal size)
    step = np.ldexp(1.0, size - 3)
    return np.clip(np.rint(y / step) * step, -TOP, TOP)


def page_exponent(top: float) -> int:
    """The least e in [E_MIN, E_MAX] with top <= 448 * 2^e."""
    e = E_MIN
    while e < E_MAX and top > TOP * 2.0**e:
        e += 1
    return e


def finite(x: np.ndarray) -> np.ndarray:
    return np.nan_to_num(np.asarray(x, dtype=np.float64), nan=0.0, posinf=BF16_MAX, neginf=-BF16_MAX)


class Page:
    """One page of one kv head, keys or values: codes (as numbers) and an exponent."""

    def __init__(self):
        self.codes, self.e = np.zeros((PAGE, DIM)), E_MIN

    def copy(self):
        p = Page()
        p.codes, p.e = self.codes.copy(), self.e
        return p

    def put(self, at: int, rows: np.ndarray) -> None:
        rows = finite(rows)
        e = page_exponent(np.abs(rows).max())
        if at > 0:
            e = max(e, self.e)
            self.codes[:at] = e4m3(self.codes[:at] * 2.0 ** (self.e - e))
        self.e = e
        self.codes[at: at + len(rows)] = e4m3(rows / 2.0**e)

    def values(self) -> np.ndarray:
        return self.codes * 2.0**self.e


class OraclePaged:
    def __init__(self, slots: int, heads: int, pages: int, max_pages: int | None = None):
        self.slots, self.heads, self.pages = slots, heads, pages
        self.max_pages = max_pages or pages
        self.lens = [0] * slots
        self.rows = [[] for _ in range(slots)]      # page ids
        self.refs = [0] * pages
        self.held = {}                              # id -> [k or v][head] Page

    def _take(self) -> int:
        p = self.refs.index(0)
        self.refs[p] = 1
        self.held[p] = [[Page() for _ in range(self.heads)] for _ in range(2)]
        return p

    def _drop(self, p: int) -> None:
        self.refs[p] -= 1
        if self.refs[p] == 0:
            del self.held[p]

    def append(self, keys, values, slots=None, counts=None) -> None:
        """keys, values [entries][heads][n][256]."""
        n = keys.shape[2]
        slots = range(keys.shape[0]) if slots is None else slots
        counts = [n] * len(slots) if counts is None else counts
        let_go = []
        for i, s in enumerate(slots):
            at, c = self.lens[s], int(counts[i])
            row = self.rows[s]
            if c and at % PAGE and self.refs[row[-1]] > 1:
                old, row[-1] = row[-1], self._take()
                self.held[row[-1]] = [[p.copy() for p in heads] for heads in self.held[old]]
                let_go.append(old)
            while len(row) * PAGE < at + c:
                row.append(self._take())
        for i, s in enumerate(slots):
            at, c = self.lens[s], int(counts[i])
            done = 0
            while done < c:
                j, inside = divmod(at + done, PAGE)
                m = min(PAGE - inside, c - done)
                for kv, x in enumerate((keys, values)):
                    for h in range(self.heads):
                        self.held[self.rows[s][j]][kv][h].put(inside, x[i, h, done: done + m])
                done += m
            self.lens[s] = at + c
        for p in let_go:
            self._drop(p)

    def trim(self, n, slots=None):
        slots = range(self.slots) if slots is None else slots
        out = []
        for s, c in zip(slots, np.broadcast_to(n, (len(slots),))):
            t = min(int(c), self.lens[s])
            self.lens[s] -= t
            while len(self.rows[s]) * PAGE - PAGE >= self.lens[s] and self.rows[s]:
                self._drop(self.rows[s].pop())
            out.append(t)
        return out

    def free(self, slots):
        self.trim(2**31 - 1, list(slots))

    def fork(self, src, dst):
        new = [(list(self.rows[s]), self.lens[s]) for s in src]
        for row, _ in new:
            for p in row:
                self.refs[p] += 1
        for d in dst:
            for p in self.rows[d]:
                self._drop(p)
        for d, (row, n) in zip(dst, new):
            self.rows[d], self.lens[d] = list(row), n

    def compact(self, pages: int | None = None) -> "OraclePaged":
        to, out = {}, OraclePaged(self.slots, self.heads, pages or self.pages, self.max_pages)
        for s in range(self.slots):
            for p in self.rows[s]:
                if p not in to:
                    to[p] = out._take()
                    out.held[to[p]] = [[x.copy() for x in heads] for heads in self.held[p]]
                    out.refs[to[p]] = 0
                out.refs[to[p]] += 1
                out.rows[s].append(to[p])
            out.lens[s] = self.lens[s]
        return out

    def values(self, slot: int):
        """keys, values [heads, len, 256] of a slot, and the values' exponents per position [heads, len]."""
        n = self.lens[slot]
        kv = [np.concatenate([np.stack([self.held[p][w][h].values() for h in range(self.heads)]) for p in self.rows[slot]], 1)[:, :n]
              if self.rows[slot] else np.zeros((self.heads, 0, DIM)) for w in range(2)]
        e = np.array([[self.held[self.rows[slot][t // PAGE]][1][h].e for t in range(n)] for h in range(self.heads)]).reshape(self.heads, n)
        return kv[0], kv[1], e


def visible(length: int, count: int, causal=True, window=0, sinks=0) -> np.ndarray:
    """[count, length]: the keys that each of the last `count` positions sees."""
    t, p = np.arange(length)[None], (length - count + np.arange(count))[:, None]
    if not causal:
        return np.ones((count, length), dtype=bool)
    see = t <= p
    return see & ((t > p - window) | (t < sinks)) if window else see


def attend(cache: OraclePaged, q, scale, slots=None, counts=None, causal=True, window=0, sinks=0):
    """(out, weight, floor, slack) [entries][q heads][n][256], in 64 bits; rows that do not exist are nan.

    out: softmax(scale q.k) . v, 0 for a query that sees nothing.
    For bounds on a kernel's rounding: weight = sum p |v| / sum p, what a relative error of every p is
    multiplied by; floor = max(p 2^e) sum |v / 2^e| / sum p over the visible keys (e: the value pages'
    exponents), what an absolute error of every weight p 2^e, relative to the largest, is multiplied by;
    slack = scale max|q| max_t sum|k_t| , what an absolute error of every query element, relative to the
    row's largest, adds to a score.
    """
    E, Hq, n, _ = q.shape
    slots = range(E) if slots is None else slots
    rep = Hq // cache.heads
    res = np.full((4, E, Hq, n, DIM), np.nan)
    for i, s in enumerate(slots):
        c = n if counts is None else int(counts[i])
        k, v, e = cache.values(s)
        see = visible(cache.lens[s], c, causal, window, sinks)
        for h in range(Hq):
            kk, vv, ee = k[h // rep], v[h // rep], e[h // rep]
            if c == 0:
                continue
            if cache.lens[s] == 0:
                res[:, i, h, :c] = 0.0
                continue
            x = np.asarray(q[i, h, :c], dtype=np.float64)
            sc = np.where(see, scale * x @ kk.T, -np.inf)
            m = sc.max(1, keepdims=True)
            p = np.where(see, np.exp(sc - np.where(np.isfinite(m), m, 0.0)), 0.0)
            l = p.sum(1, keepdims=True)
            l1 = np.where(l > 0, l, 1.0)
            res[0, i, h, :c] = p @ vv / l1
            res[1, i, h, :c] = p @ np.abs(vv) / l1
            res[2, i, h, :c] = (p * 2.0**ee).max(1, keepdims=True) * (see @ np.abs(vv / 2.0 ** ee[:, None])) / l1
            ksum = np.where(see, np.abs(kk).sum(1)[None], 0.0).max(1, keepdims=True)
            res[3, i, h, :c] = abs(scale) * np.abs(x).max(1, keepdims=True) * ksum
    return res
