"""Plain references of the paged KV cache: its page calls as Python loops over lists, and attention by its
definition in 64 bits, row by row.  No code of the package."""
import math

import numpy as np

CAPACITY, INVALID = 1, 8


class Book:
    """tables, lengths and reference counts, as vc.h describes the page calls"""

    def __init__(self, pages, page, seqs, columns, window, sinks):
        self.pages, self.page, self.seqs, self.columns, self.window, self.sinks = pages, page, seqs, columns, window, sinks
        self.table = [[-1] * columns for _ in range(seqs)]
        self.len = [0] * seqs
        self.refs = [0] * pages
        self.status = 0
        self.copies = []       # (source page, destination page, positions)

    def _up(self, n):
        return -(-n // self.page)

    def _release(self, s, col):
        e = self.table[s][col]
        if e >= 0:
            self.refs[e] -= 1
            self.table[s][col] = -1

    def _free(self):
        return [p for p in range(self.pages) if self.refs[p] == 0]

    def resize(self, seqs, targets):
        """-> pos; targets: the lengths asked for"""
        page, most = self.page, self.columns * self.page
        rows, named = [], set()
        for s, to in zip(seqs, targets):
            ok = 0 <= s < self.seqs and s not in named and to >= 0
            if 0 <= s < self.seqs:
                named.add(s)
            if ok:
                at = min(self.len[s], to)
                ok = at % page == 0 or self.table[s][at // page] >= 0
            rows.append((s, self.len[s], to) if ok else None)
        for r in rows:
            if r is None:
                continue
            s, have, to = r
            for col in range(self._up(min(to, most)), self._up(have)):
                self._release(s, col)
            start = min(have, to)
            if self.window:
                for col in range(self._up(self.sinks), self.columns):
                    if (col + 1) * page - 1 <= start - self.window:
                        self._release(s, col)
        plans, asked, free = [], 0, self._free()
        for r in rows:
            cols = []
            if r and r[1] < r[2] <= most:
                s, have, to = r
                if have % page and self.refs[self.table[s][have // page]] > 1:
                    cols.append(have // page)
                cols += range(self._up(have), self._up(to))
            plans.append((asked, cols))
            asked += len(cols)
        pos = []
        for r, (first, cols) in zip(rows, plans):
            if r is None or r[2] > most or (cols and first + len(cols) > len(free)):
                self.status |= INVALID if r is None else CAPACITY
                pos.append(-1)
                continue
            s, have, to = r
            for k, col in enumerate(cols):
                new = free[first + k]
                if col < self._up(have):
                    old = self.table[s][col]
                    self.refs[old] -= 1
                    self.copies.append((old, new, have % page))
                self.table[s][col] = new
                self.refs[new] = 1
            self.len[s] = to
            pos.append(min(have, to))
        return pos

    def fork(self, src, dst):
        """-> done"""
        good, named = [], set()
        for s, d in zip(src, dst):
            good.append(0 <= s < self.seqs and 0 <= d < self.seqs and d not in named and d not in src)
            if 0 <= d < self.seqs:
                named.add(d)
        for ok, d in zip(good, dst):
            if ok:
                for col in range(self._up(self.len[d])):
                    self._release(d, col)
        free, asked, done = self._free(), 0, []
        for ok, s, d in zip(good, src, dst):
            if not ok:
                self.status |= INVALID
                done.append(0)
                continue
            have = self.len[s]
            part = have % self.page != 0 and self.table[s][have // self.page] >= 0
            k = asked
            asked += part
            if part and k >= len(free):
                self.status |= CAPACITY
                self.len[d] = 0
                done.append(0)
                continue
            for col in range(have // self.page):
                e = self.table[s][col]
                if e >= 0:
                    self.table[d][col] = e
                    self.refs[e] += 1
            if part:
                self.table[d][have // self.page] = free[k]
                self.refs[free[k]] = 1
                self.copies.append((self.table[s][have // self.page], free[k], have % self.page))
            self.len[d] = have
            done.append(1)
        return done

    def compact(self):
        """-> the pages in use, [(from, to)]"""
        live = [p for p in range(self.pages) if self.refs[p] > 0]
        n = len(live)
        moves = list(zip([p for p in live if p >= n], [p for p in range(n) if self.refs[p] == 0]))
        name = dict(moves)
        self.table = [[name.get(e, e) for e in row] for row in self.table]
        for a, b in moves:
            self.refs[b], self.refs[a] = self.refs[a], 0
        return n, moves


def attend_row(q, keys, values, seen, scale):
    """one query's output in 64 bits over the keys that it sees, and what its error bounds need: sum w |v| / sum w,
    the largest sum |q k| scale, and sum |v| over the seen keys"""
    if not seen.any():
        z = np.zeros(values.shape[1])
        return z, z, 0.0, z
    k, v = keys[seen].astype(np.float64), values[seen].astype(np.float64)
    z = k @ q.astype(np.float64) * scale
    w = np.exp(z - z.max())
    w /= w.sum()
    return w @ v, w @ np.abs(v), float((np.abs(k) @ np.abs(q.astype(np.float64)) * abs(scale)).max()), np.abs(v).sum(0)


def tolerance(ref, abs_weighted, dots, abs_seen, n_dims, half_step, weight_floor):
    """|error| of an output whose scores are summed in fp32, whose weights are rounded once to 16 bits (relative
    half_step, and weight_floor absolutely below the type's normal range; the largest weight is 1) and whose value is
    rounded once:
      scores: at most n_dims + 2 roundings of 2^-24 of sum |q k| scale, and 2^-21 for exp2 and its argument's
        rounding (|z| 2^-24 log2 e, |z| <= dots), in the weights above and below the quotient: a factor 2
      the sums over keys in fp32 and the joins of key ranges: 2^-18 of sum w |v| (up to 2^6 roundings in a chain)."""
    weights = 2.0 * ((n_dims + 4) * 2.0 ** -24 * dots + 2.0 ** -21) + 2.0 ** -18
    err = (half_step + weights) * abs_weighted + weight_floor * abs_seen
    return err + half_step * (np.abs(ref) + err) + weight_floor


HALF_STEP = {"bf16": 2.0 ** -8, "fp16": 2.0 ** -11}
# half a step of the smallest numbers: fp16's subnormals; bf16's weights below fp32's range are 0 (2^-126)
FLOOR = {"bf16": 2.0 ** -126, "fp16": 2.0 ** -25}


def seen_keys(p, n, window, sinks):
    t = np.arange(n)
    ok = t <= p
    if window:
        ok &= (t < sinks) | (t > p - window)
    return ok


def default_scale(head_dim):
    return 1.0 / math.sqrt(head_dim)
