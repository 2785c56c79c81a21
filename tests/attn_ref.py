"""Plain 64-bit forms of the attention and cache operators, for their tests.

Attention: one query at a time over the list of keys that it sees.  The cache:
lists and dicts on the host, changed token by token."""
from __future__ import annotations

import numpy as np


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


def attend(q, k, v, seen, scale):
    """q [D], k and v [m, D] float64, seen bool [m] -> (o [D], A [D], reach):
    o the attention output, A = sum w |v|, reach = max over the seen keys of
    scale * sum |q k| (0 where nothing is seen)."""
    if not seen.any():
        return np.zeros_like(q), np.zeros_like(q), 0.0
    ks, vs = k[seen], v[seen]
    with np.errstate(all="ignore"):
        s = scale * (ks @ q)
        w = np.exp(s - s.max())
        w /= w.sum()
        # reach bounds the error of finite scores
        reach = scale * np.nanmax(np.abs(ks) @ np.abs(q), initial=0.0)
        return w @ vs, w @ np.abs(vs), float(reach if np.isfinite(reach) else 0.0)


# Rounding of an output o = sum w v / sum w against its exact value, with
# A = sum w |v| / sum w, u the unit roundoff of the element type:
# (11 and 8 bits of significand: u = 2^-11 and 2^-8),
#   u |o|              the output's rounding                        (<= u A)
#   u A                the weights' rounding before the product with v
#   2 e A              e = relative error of a weight from its fp32 score: the
#                      score's sum of D products, (D + 2) 2^-24 reach, the
#                      scaling and subtraction of the maximum, 4 2^-24 reach,
#                      and the exponential, 2^-22; once in numerator and sum
#   fp32 sums          (keys + 64) 2^-24 A covers the accumulations
# and for fp16 weights below 2^-24 of the largest (subnormal after the lift of
# 2^10) an absolute 2^-35 per key times max |v|, and subnormal outputs 2^-25.
def tolerance(A, reach, keys, D, dtype, vmax):
    u = 2.0 ** -11 if dtype == "f16" else 2.0 ** -8
    e = (D + 6) * 2.0 ** -24 * reach + 2.0 ** -22
    tol = (2 * u + 2 * e + (keys + 64) * 2.0 ** -24) * A
    if dtype == "f16":
        tol = tol + keys * 2.0 ** -35 * vmax + 2.0 ** -25
    return tol + 1e-30


def check(out, want, A, reach, keys, D, dtype, vmax, what):
    """out against want, NaN and infinities in the same places."""
    fine = np.isfinite(want)
    assert np.array_equal(np.isfinite(out), fine), f"{what}: {(np.isfinite(out) != fine).sum()} values (not) finite"
    err = np.abs(out - want)[fine]
    tol = np.broadcast_to(tolerance(A, reach, keys, D, dtype, vmax), want.shape)[fine]
    bad = err > tol
    assert not bad.any(), f"{what}: {bad.sum()} of {bad.size} off, worst {np.max(err / tol):.3g} of the tolerance"


class Model:
    """The cache's bookkeeping and contents: rows of token ids in pages."""

    def __init__(self, pages, page, rows, width):
        self.page, self.width = page, width
        self.tables = [[-1] * width for _ in range(rows)]
        self.lens = [0] * rows
        self.refs = [0] * pages
        self.slots = {}  # (page, slot) -> token
        self.status = 0

    def tokens(self, b):
        return [self.slots.get((self.tables[b][p // self.page], p % self.page)) for p in range(self.lens[b])]

    def _free(self):
        return [p for p, r in enumerate(self.refs) if r == 0]

    def reserve(self, add):
        pos, need = [], []
        for b, n in enumerate(add):
            if n < 0:
                need.append(None)
                self.status |= 4
            elif self.lens[b] + n > self.width * self.page:
                need.append(None)
                self.status |= 2
            else:
                need.append(-(-(self.lens[b] + n) // self.page) - -(-self.lens[b] // self.page))
        free, used = self._free(), 0
        for b, n in enumerate(add):
            if need[b] is None:
                pos.append(-1)
                continue
            used += need[b]
            if need[b] and used > len(free):
                self.status |= 1
                pos.append(-1)
                continue
            have = -(-self.lens[b] // self.page)
            for i in range(need[b]):
                p = free[used - need[b] + i]
                self.tables[b][have + i] = p
                self.refs[p] = 1
            pos.append(self.lens[b])
            self.lens[b] += n
        return pos

    def write(self, pos, add, ids):
        at = 0
        for b, n in enumerate(add):
            for i in range(n):
                if pos[b] >= 0:
                    p = pos[b] + i
                    self.slots[self.tables[b][p // self.page], p % self.page] = ids[at]
                at += 1

    def fork(self, parents):
        rows = len(self.tables)
        par = []
        for p in parents:
            if not -1 <= p < rows:
                self.status |= 4
            par.append(p if 0 <= p < rows else -1)
        for b in range(rows):
            for i in range(-(-self.lens[b] // self.page)):
                full = (i + 1) * self.page <= self.lens[b]
                self.refs[self.tables[b][i]] += par.count(b) - 1 if full else min(0, par.count(b) - 1)
        tables, lens, wants = [], [], []
        for i, p in enumerate(par):
            row, n = [-1] * self.width, 0
            if p >= 0:
                n = self.lens[p]
                row[:-(-n // self.page)] = self.tables[p][:-(-n // self.page)]
                if n % self.page and p in par[:i]:
                    wants.append((i, n // self.page, row[n // self.page]))
                    row[n // self.page] = -1
            tables.append(row)
            lens.append(n)
        free = self._free()
        for k, (i, slot, old) in enumerate(wants):
            if k < len(free):
                tables[i][slot] = free[k]
                self.refs[free[k]] = 1
                for s in range(lens[i] % self.page):
                    self.slots[free[k], s] = self.slots[old, s]
            else:
                lens[i] = slot * self.page
                self.status |= 1
        self.tables, self.lens = tables, lens

    def compact(self, pos, keep, count):
        refs = list(self.refs)  # the decisions are taken before anything changes
        go = []
        for b, (p, c) in enumerate(zip(pos, count)):
            go.append(False)
            if p < 0:
                self.status |= 4 if p < -1 else 0
                continue
            n, ks = self.lens[b], keep[b][:max(c, 0)]
            if not 0 <= c <= len(keep[b]) or p > n or any(not 0 <= k < n - p for k in ks) or sorted(set(ks)) != list(ks):
                self.status |= 4
                continue
            end = p + c
            touched = {(p + j) // self.page for j, k in enumerate(ks) if j != k}
            if end % self.page:
                touched.add(end // self.page)
            if any(refs[self.tables[b][i]] > 1 for i in touched):
                self.status |= 8
                continue
            go[b] = True
        for b, ok in enumerate(go):
            if not ok:
                continue
            at = lambda p: (self.tables[b][p // self.page], p % self.page)  # noqa: E731
            moved = [self.slots.get(at(pos[b] + k)) for k in keep[b][:count[b]]]
            for j, t in enumerate(moved):
                self.slots[at(pos[b] + j)] = t
            end = pos[b] + count[b]
            for i in range(-(-end // self.page), -(-self.lens[b] // self.page)):
                self.refs[self.tables[b][i]] -= 1
                self.tables[b][i] = -1
            self.lens[b] = end
