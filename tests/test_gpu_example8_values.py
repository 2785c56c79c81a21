"""The example's serving loop over a cache of 8 bits, followed call by call: what the cache holds after forks, trees and
compaction are the tokens that were appended, and attention is that over what it holds."""
import numpy as np
import pytest

from tests import attn_ref, kv8_ref
from tests.gpu_util import say, torch

pytestmark = pytest.mark.gpu

q = pytest.importorskip("gemm_unpack_bit_amd")

# A key or value in the cache against the exact one x (rotated in 64 bits): rounding to 4 significant bits, 2^-4 |x| at
# most; of subnormal codes half a step, 2^-10 2^e, where the block's largest value m is more than 224 * 2^e (its exponent is
# the least that holds m), so less than 2^-17 m, once when it was written and once for each time the exponent grew, each
# time at most half of the last: 2^-16 m; and the rotation in 32 bits, (|a| + |b|) (2^-20 + 2^-22) <= 2^-18 m, rounded
# with the rest.  m is at most the largest value so far.
RELATIVE, OF_LARGEST = 2.0 ** -4, 2.0 ** -16 + 2.0 ** -17


class Follow:
    """The example's calls, each beside a plain model: of every cache, layer and row the exact keys and values."""

    def __init__(self, monkeypatch):
        self.rows = {}  # id(cache) -> [layer][row] -> list of (key, value)
        self.caches, self.largest, self.seen = [], 0.0, 0
        self.true = {n: getattr(q, n) for n in ("kv_append", "kv_read", "kv_fork", "kv_compact", "attn_tree")}
        for n in self.true:
            monkeypatch.setattr(q, n, getattr(self, n))

    def of(self, cache):
        if id(cache) not in self.rows:
            self.rows[id(cache)] = [[[] for _ in range(cache.rows)] for _ in range(cache.k.shape[0])]
            self.caches.append(cache)  # (kept, so that no other takes its place)
        return self.rows[id(cache)]

    def kv_append(self, cache, layer, k, v, cu, pos, q=None, freqs=None, at=None, **more):
        keys, values = attn_ref.f64(k), attn_ref.f64(v)
        keys = kv8_ref.rotate(keys, at.cpu().numpy(), freqs.cpu().numpy(), False)
        self.largest = max(self.largest, np.abs(keys).max(), np.abs(values).max())
        ends = cu.tolist()
        for b, p in enumerate(pos.tolist()):
            row = self.of(cache)[layer][b]
            assert p == len(row)
            row += list(zip(keys[ends[b]:ends[b + 1]], values[ends[b]:ends[b + 1]]))
        return self.true["kv_append"](cache, layer, k, v, cu, pos, q=q, freqs=freqs, at=at, **more)

    def held(self, cache, layer):
        """The cache's rows, compared with the model's: [row] -> keys, values [tokens, heads, dim]."""
        t, rows = torch(), self.of(cache)[layer]
        lens = cache.lens.tolist()
        assert lens == [len(r) for r in rows]
        cu = np.concatenate([[0], np.cumsum(lens)])
        ints = lambda a: t.tensor([int(i) for i in a], dtype=t.int32, device="cuda")  # noqa: E731
        k, v = self.true["kv_read"](cache, layer, ints(cu), ints([0] * len(lens)), tokens=int(cu[-1]))
        out = []
        for b, row in enumerate(rows):
            got = [attn_ref.f64(x[cu[b]:cu[b + 1]]) for x in (k, v)]
            for g, want in zip(got, zip(*row)):
                want = np.array(want)
                assert (np.abs(g - want) <= RELATIVE * np.abs(want) + OF_LARGEST * self.largest).all(), (layer, b)
            self.seen += len(row)
            out.append(got)
        return out

    def kv_read(self, cache, layer, cu, start, **more):
        k, v = self.true["kv_read"](cache, layer, cu, start, **more)
        assert start.tolist() == [0] * cache.rows
        for x, of in ((k, 0), (v, 1)):
            want = np.concatenate([r[of] for r in self.held(cache, layer)])
            assert np.array_equal(attn_ref.f64(x), want)
        return k, v

    def kv_fork(self, cache, parents, out=None):
        new = self.true["kv_fork"](cache, parents, out)
        self.of(new)[:] = [[list(layer[p]) if p >= 0 else [] for p in parents.tolist()] for layer in self.of(cache)]
        return new

    def kv_compact(self, cache, pos, keep, count):
        where, keeps, counts = pos.tolist(), keep.tolist(), count.tolist()
        self.true["kv_compact"](cache, pos, keep, count)
        for layer in self.of(cache):
            for b, p in enumerate(where):
                layer[b][p:] = [layer[b][p + i] for i in keeps[b][:counts[b]]]

    def attn_tree(self, x, cache, layer, cu, pos, mask=None, **more):
        out = self.true["attn_tree"](x, cache, layer, cu, pos, mask, **more)
        ends, heads, dim = cu.tolist(), x.shape[1], x.shape[2]
        xs, got = attn_ref.f64(x), attn_ref.f64(out)
        words = None if mask is None else mask.cpu().numpy().view(np.uint64)
        for b, (k, v) in enumerate(self.held(cache, layer)):
            for i in {ends[b], ends[b + 1] - 1}:  # a row's first and last token
                n, n0 = len(k), len(k) - (ends[b + 1] - ends[b])
                seen = np.arange(n) <= n0 + i - ends[b] if words is None else np.arange(n) < n0
                for j in range(n - n0 if words is not None else 0):
                    seen[n0 + j] = bool(int(words[i, 0]) >> j & 1)
                for h in range(heads):
                    kk, vv = k[:, h // (heads // k.shape[1])], v[:, h // (heads // k.shape[1])]
                    o, A, reach = attn_ref.attend(xs[i, h], kk, vv, seen, dim ** -0.5)
                    attn_ref.check(got[i, h], o, A, reach, n, dim, "f16", np.abs(vv).max(), f"layer {layer} row {b} token {i} head {h}")
        return out


@pytest.mark.parametrize("seed,lengths,ahead", [(1, (37, 5, 120), 4), (3, (1, 16, 64, 3), 7)])
def test_decode_layers_over_a_cache_of_8_bits(seed, lengths, ahead, monkeypatch):
    from examples import decode_layers as ex

    say("decode_layers8, followed", seed, lengths, ahead)
    f = Follow(monkeypatch)
    r = ex.main(seed, lengths, ahead, cache_type=torch().float8_e4m3fn)
    assert r["status"] == 0 and f.seen > 20 * sum(lengths)
    # Each way rounds keys and values to 4 significant bits, a relative 2^-4 at most, in every layer, and the rest as with
    # a cache of 16 bits.
    assert r["difference"] < 2 * (2 * ex.LAYERS * 2.0 ** -4 + (8 * ex.LAYERS + 2) * 2.0 ** -11)
