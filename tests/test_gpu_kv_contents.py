"""GPU tests of what the cache's calls move, element by element: every 16 bits of a
token's keys and values are random and its own, in every layer and head."""
import numpy as np
import pytest

from tests.attn_ref import Model
from tests.gpu_util import say, torch

pytestmark = pytest.mark.gpu

q_ = pytest.importorskip("gemm_unpack_bit_amd")


def _dev(a):
    return torch().from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()


def _cu(n):
    return _dev(np.concatenate([[0], np.cumsum(n)]))


class Cache:
    """A cache beside the model; token id i has the bits store[0 or 1, layer, i] (heads by elements)."""

    def __init__(self, layers, pages, page, kv, D, rows, width, dtype, seed, source):
        t = torch()
        self.rng, self.t, self.dtype, self.source = np.random.default_rng(seed), t, dtype, source
        self.cache = q_.KvCache.empty(layers, pages, page, kv, D, rows, width, dtype=dtype)
        for pool in (self.cache.k, self.cache.v):
            pool.view(t.int16).random_(-2 ** 15, 2 ** 15)
        self.model = Model(pages, page, rows, width)
        self.store = np.zeros((2, layers, 0, kv, D), np.int16)

    def _as(self, x):
        """[tokens, heads, D] bits -> an array of the layout that is tested."""
        t = self.t
        x = t.from_numpy(x).cuda().view(self.dtype)
        n, h, d = x.shape
        if self.source == "heads outside":
            return x.transpose(0, 1).contiguous().transpose(0, 1)
        if self.source == "padded heads":
            out = t.zeros(n, h, d + 24, dtype=self.dtype, device="cuda")[:, :, 8:8 + d]
        elif self.source == "fused":
            out = t.zeros(n, 3 * h + 1, d, dtype=self.dtype, device="cuda")[:, h + 1:2 * h + 1]
        else:
            return x
        out.copy_(x)
        return out

    def append(self, add):
        c, n, first = self.cache, sum(add), self.store.shape[2]
        pos = q_.kv_reserve(c, _cu(add))
        want = self.model.reserve(add)
        assert pos.tolist() == want
        new = self.rng.integers(-2 ** 15, 2 ** 15, (2, self.store.shape[1], n) + self.store.shape[3:], dtype=np.int16)
        self.store = np.concatenate([self.store, new], 2)
        for layer in range(new.shape[1]):
            k, v = self._as(new[0, layer]), self._as(new[1, layer])
            assert n == 0 or self.t.equal(k.contiguous().view(self.t.int16).cpu(), self.t.from_numpy(new[0, layer]))
            before = [p[:layer].clone().view(self.t.int16) for p in (c.k, c.v)]
            q_.kv_write(c, layer, k, v, _cu(add), pos)
            for p, b in zip((c.k, c.v), before):
                assert self.t.equal(p[:layer].view(self.t.int16), b), "another layer was written"
        self.model.write(want, add, list(range(first, first + n)))
        self.check("append")
        return want

    def check(self, what):
        c, m = self.cache, self.model
        assert (c.lens.tolist(), c.refs.tolist(), c.tables.tolist()) == (m.lens, m.refs, m.tables), what
        for i, pool in enumerate((c.k, c.v)):
            bits = pool.view(self.t.int16).flatten(1, 2).cpu().numpy()  # [layers, pages * page, heads, D]
            for b in range(len(m.lens)):
                at = [m.tables[b][p // m.page] * m.page + p % m.page for p in range(m.lens[b])]
                if at:
                    assert np.array_equal(bits[:, at], self.store[i][:, m.tokens(b)]), f"{what}: row {b}, {'kv'[i]}"


@pytest.mark.parametrize("kv,D,page", [(1, 64, 16), (3, 64, 32), (5, 128, 16), (8, 128, 64), (2, 64, 256)])
@pytest.mark.parametrize("source,dtype", [("plain", "float16"), ("heads outside", "bfloat16"), ("padded heads", "float16"),
                                          ("fused", "bfloat16")])
def test_every_element_goes_where_its_token_goes(kv, D, page, source, dtype):
    t = torch()
    say("kv contents", kv, D, page, source, dtype)
    rows, layers = 6, 3
    x = Cache(layers, 60, page, kv, D, rows, 8, getattr(t, dtype), kv + page, source)
    rng = x.rng
    x.append([page + 3, 5, 0, 2 * page, page - 1, 1])
    x.append([1, 1, 1, 1, 1, 1])
    x.model.fork([0, 0, 1, 3, 0, 1])  # copies of partial pages, a full one shared
    x.cache = q_.kv_fork(x.cache, _dev([0, 0, 1, 3, 0, 1]))
    x.check("fork")
    add = [7, 13, 9, 20, 1, 11]
    pos = x.append(add)
    keep = [sorted(rng.choice(n, max(n // 2, 1), replace=False).tolist()) for n in add]
    count = [len(k) for k in keep]
    keep = [k + [0] * (10 - len(k)) for k in keep]
    x.model.compact(pos, keep, count)
    q_.kv_compact(x.cache, _dev(pos), _dev(keep), _dev(count))
    x.check("compact")
    x.append([2, 0, 3, 1, 0, 4])
    x.model.fork([5, 4, 4, -1, 0, 2, 1, 0, 3])  # more rows than before
    x.cache = q_.kv_fork(x.cache, _dev([5, 4, 4, -1, 0, 2, 1, 0, 3]))
    x.check("fork of more rows")
    assert int(x.cache.status) == x.model.status == 0


@pytest.mark.parametrize("kv,D", [(3, 64), (2, 128)])
def test_elements_through_the_calls_of_many_workgroups(kv, D):
    """Enough rows for the fork of several launches, and kept tokens by the hundred."""
    t = torch()
    say("kv contents, many rows", kv, D)
    rows = 280
    x = Cache(2, 2600, 16, kv, D, rows, 24, t.float16, 11, "fused")
    x.append([int(n) for n in x.rng.integers(0, 40, rows)])
    parents = [int(p) for p in x.rng.integers(-1, rows, rows)]
    x.model.fork(parents)
    x.cache = q_.kv_fork(x.cache, _dev(parents))
    x.check("fork")
    add = [int(n) for n in x.rng.integers(0, 12, rows)]
    add[3] = 200
    pos = x.append(add)
    assert int(x.cache.status) == 0
    keep = [sorted(x.rng.choice(n, n - n // 3, replace=False).tolist()) for n in add]
    count, most = [len(k) for k in keep], max(len(k) for k in keep)
    keep = [k + [-1] * (most - len(k)) for k in keep]
    x.model.compact(pos, keep, count)
    q_.kv_compact(x.cache, _dev(pos), _dev(keep), _dev(count))
    x.check("compact")
