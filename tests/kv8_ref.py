"""Plain 64-bit forms of the 8-bit cache: e4m3 codes with a power of two per
block of 16 tokens and head, and of the position rotation, for their tests."""
from __future__ import annotations

import numpy as np

BLOCK = 16
CODES = np.array([(-1.0 if c & 128 else 1.0) * ((c & 7) * 2.0 ** -9 if not c >> 3 & 15 else (8 + (c & 7)) * 2.0 ** ((c >> 3 & 15) - 10))
                  for c in range(256)])
CODES[[127, 255]] = np.nan


def values(codes, exps):
    """codes uint8 [..., page_size, heads, dim], exps uint8 [..., page_size / 16, heads] -> float64."""
    return CODES[codes] * 2.0 ** (np.repeat(exps, BLOCK, axis=-2).astype(np.float64) - 127)[..., None]


def step(x, e):
    """The distance of neighbouring codes at x under the exponent byte e (of the binade of |x|)."""
    with np.errstate(divide="ignore"):
        top = np.floor(np.log2(np.abs(x) * 2.0 ** (127.0 - e)))
    return 2.0 ** (np.maximum(top, -6) - 3 + e - 127.0)


def rounded(x, e):
    """x to the nearest code's value under e, even ones at ties (NaN stays)."""
    s = step(np.nan_to_num(x), e)
    return np.round(x / s) * s


def exponent(most):
    """The exponent byte of a block whose largest finite |x| is `most`."""
    m, x = np.frexp(most)  # m 2^x, 1/2 <= m < 1; 448 = 0.875 2^9
    e = np.where(m > 0.875, x - 8, x - 9)
    return np.maximum(np.where(most > 0, e, -64), -64) + 127


def rotate(x, at, freqs, interleaved):
    """x [tokens, heads, dim] turned by the angles at[t] * freqs[i]."""
    y, n = x.copy(), len(freqs)
    if n:
        angle = (at.astype(np.float64)[:, None] * freqs.astype(np.float64))[:, None, :]
        i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
        a, b = x[..., i], x[..., j]
        y[..., i], y[..., j] = a * np.cos(angle) - b * np.sin(angle), a * np.sin(angle) + b * np.cos(angle)
    return y


def turn_error(x, freqs, interleaved):
    """Bound of the rotation's error in 32 bits: (|a| + |b|) times the error of a sine or cosine (the angle's fraction of
    a turn rounded to 2^-25, times 2 pi; the function's 2^-21) and of two products and a sum (3 * 2^-24)."""
    y, n = np.zeros_like(x), len(freqs)
    if n:
        i, j = (slice(0, 2 * n, 2), slice(1, 2 * n, 2)) if interleaved else (slice(0, n), slice(n, 2 * n))
        both = (np.abs(x[..., i]) + np.abs(x[..., j])) * (2.0 ** -20 + 2.0 ** -22)
        y[..., i] = y[..., j] = both
    return y


class Pool:
    """One pool (keys or values) of a cache of 8 bits: values and exponents, [layers, tokens, heads(, dim)]."""

    def __init__(self, codes, exps):
        layers, pages, page, heads, dim = codes.shape
        self.page = page
        self.v = values(codes, exps).reshape(layers, pages * page, heads, dim)
        self.e = exps.astype(np.int64).reshape(layers, -1, heads)

    def place(self, table, p):
        return table[p // self.page] * self.page + p % self.page

    def append(self, layer, table, pos, new):
        """new [n, heads, dim] to positions pos ... of the row; returns [(place, exact value before rounding)]."""
        n, out = len(new), []
        for first in range(pos // BLOCK * BLOCK, pos + n, BLOCK):
            places = [self.place(table, p) for p in range(first, min(first + BLOCK, pos + n))]
            block, old = places[0] // BLOCK, max(0, pos - first)
            fresh = new[max(0, first - pos):first - pos + BLOCK]
            fresh = np.where(np.isfinite(fresh), fresh, np.nan)
            e = exponent(np.nanmax(np.nan_to_num(np.abs(fresh)), axis=(0, 2)))
            if old:
                had = self.e[layer, block]
                e = np.maximum(e, had)
                self.v[layer, places[:old]] = rounded(self.v[layer, places[:old]], e[None, :, None])
            self.e[layer, block] = e
            self.v[layer, places[old:]] = rounded(fresh, e[None, :, None])
            out += list(zip(places[old:], fresh))
        return out

    def copy(self, src_page, dst_page, tokens):
        a, b, p = src_page * self.page, dst_page * self.page, self.page
        self.v[:, b:b + tokens] = self.v[:, a:a + tokens]
        k = -(-tokens // BLOCK)
        self.e[:, b // BLOCK:b // BLOCK + k] = self.e[:, a // BLOCK:a // BLOCK + k]
        assert k <= p // BLOCK

    def compact(self, table, pos, kept):
        end = pos + len(kept)
        for first in range(pos // BLOCK * BLOCK, end, BLOCK):
            to = list(range(first, min(first + BLOCK, end)))
            come = [p if p < pos else pos + kept[p - pos] for p in to]
            if come == to:
                continue
            src, dst = [self.place(table, p) for p in come], [self.place(table, p) for p in to]
            e = np.max(self.e[:, [s // BLOCK for s in src]], axis=1)
            self.v[:, dst] = rounded(self.v[:, src], e[:, None, :, None])
            self.e[:, dst[0] // BLOCK] = e
