"""GPU tests of the paged cache's calls against a model on the host
(tests/attn_ref.py): tables, lengths, reference counts, status bits and contents
have to be equal after every call."""
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


class Both:
    """A cache on the GPU beside the model.  Token id i has keys i + 0.25 * layer (value: negated) in every place."""

    def __init__(self, layers, pages, page, kv, D, rows, width, dtype):
        t = torch()
        self.cache = q_.KvCache.empty(layers, pages, page, kv, D, rows, width, dtype=dtype)
        self.cache.k.fill_(-1)
        self.cache.v.fill_(-1)
        self.model = Model(pages, page, rows, width)
        self.ids, self.dtype, self.t = 0, dtype, t

    def append(self, add):
        t, c = self.t, self.cache
        want = self.model.reserve(add)
        pos = q_.kv_reserve(c, _cu(add))
        assert pos.tolist() == want
        n = sum(add)
        ids = [(self.ids + i) % 200 for i in range(n)]
        self.ids += n
        base = t.tensor(ids, dtype=t.float32, device="cuda")[:, None, None].expand(n, c.heads_kv, c.head_dim)
        for layer in range(c.k.shape[0]):
            wide = t.zeros(n, 2 * c.heads_kv + 1, c.head_dim, dtype=self.dtype, device="cuda")  # strided rows
            wide[:, :c.heads_kv] = (base + 0.25 * layer).to(self.dtype)
            wide[:, c.heads_kv:2 * c.heads_kv] = -(base + 0.25 * layer).to(self.dtype)
            q_.kv_write(c, layer, wide[:, :c.heads_kv], wide[:, c.heads_kv:2 * c.heads_kv], _cu(add), pos)
        self.model.write(want, add, ids)
        self.check("append")
        return want

    def fork(self, parents):
        self.model.fork(parents)
        self.cache = q_.kv_fork(self.cache, _dev(parents))
        self.check(f"fork {parents}")

    def compact(self, pos, keep, count):
        self.model.compact(pos, keep, count)
        q_.kv_compact(self.cache, _dev(pos), _dev(keep).view(len(pos), -1), _dev(count))
        self.check(f"compact {pos} {keep} {count}")

    def check(self, what):
        c, m = self.cache, self.model
        assert c.lens.tolist() == m.lens, what
        assert c.refs.tolist() == m.refs, what
        assert c.tables.tolist() == m.tables, what
        assert int(c.status) == m.status, what
        k, v = c.k.float(), c.v.float()
        for b in range(len(m.lens)):
            want = m.tokens(b)
            if not want:
                continue
            at = self.t.tensor([m.tables[b][p // m.page] * m.page + p % m.page for p in range(m.lens[b])], device="cuda")
            for layer in range(k.shape[0]):
                w = self.t.tensor(want, device="cuda")[:, None, None] + 0.25 * layer
                w = w.to(self.dtype).float()
                got = k[layer].reshape(-1, c.heads_kv, c.head_dim)[at]
                assert bool((got == w).all()), f"{what}: keys of row {b} layer {layer}"
                got = v[layer].reshape(-1, c.heads_kv, c.head_dim)[at]
                assert bool((got == -w).all()), f"{what}: values of row {b} layer {layer}"


@pytest.mark.parametrize("page,kv,D,rows,dtype", [(16, 2, 64, 5, "float16"), (32, 1, 128, 9, "float16"),
                                                  (128, 3, 64, 3, "float16"), (16, 8, 128, 70, "float16"),
                                                  (16, 1, 64, 300, "float16")])
def test_random_life(page, kv, D, rows, dtype):
    """Appends, trees with their compaction and forks in random order, from an empty pool to a full one."""
    t = torch()
    rng = np.random.default_rng(page + rows)
    x = Both(3, 3 * rows + 4, page, kv, D, rows, 5, getattr(t, dtype))
    say("kv life", page, kv, D, rows)
    for step in range(14):
        kind = step % 3
        if kind == 0:
            x.append(rng.integers(0, page + 3, rows).tolist())
        elif kind == 1:
            add = rng.integers(0, 24, rows).tolist()
            pos = x.append(add)
            M, keep, count = 7, [], []
            for b in range(rows):
                n = add[b] if pos[b] >= 0 else 0
                c = int(rng.integers(0, min(n, M) + 1))
                keep.append(sorted(rng.choice(n, c, replace=False).tolist()) + [-1] * (M - c) if n else [-1] * M)
                count.append(c if pos[b] >= 0 else 0)
            x.compact(pos, keep, count)
        else:
            x.fork([int(p) for p in rng.integers(-1, rows, rows)])
    # free everything: all references go
    x.compact([0] * rows, [[]] * rows, [0] * rows)
    assert sum(x.model.refs) == 0


def test_pages_run_out():
    """Rows in order get pages while there are any; others stay as they were, and say so."""
    t = torch()
    say("kv full pool")
    x = Both(2, 6, 16, 2, 64, 4, 4, t.float16)
    assert x.append([20, 16, 33, 1]) == [0, 0, 0, -1]       # 2 + 1 + 3 pages, and none for the last row
    assert int(x.cache.status) == q_.KV_NO_PAGES
    x.model.status = 0
    x.cache.status.zero_()
    assert x.append([12, 0, 5, 0]) == [20, 16, 33, 0]       # inside pages that they have
    assert x.append([70, 0, 0, 0])[0] == -1                 # the table is too short
    assert int(x.cache.status) == q_.KV_TABLE_FULL
    x.fork([0, 0, 1, 2])                                    # shares full pages
    x.fork([3, 3, 3, 3])                                    # three copies: the last pages
    x.fork([0, -1, 9, -5])                                  # parents out of range count as none
    assert int(x.cache.status) == q_.KV_TABLE_FULL | q_.KV_BAD_INDEX
    y = Both(2, 4, 16, 2, 64, 4, 4, t.float16)
    y.append([20, 0, 0, 0])
    y.fork([0, 0, 0, 0])                                    # two copies, then the last child keeps its full page only
    assert y.cache.lens.tolist() == [20, 20, 20, 16] and int(y.cache.status) == q_.KV_NO_PAGES


def test_compaction_refusals_leave_the_row():
    t = torch()
    say("kv compact refusals")
    x = Both(1, 40, 16, 1, 64, 4, 6, t.float16)
    x.append([16, 20, 40, 10])
    x.append([24, 8, 8, 8])
    x.fork([0, 0, 2, 3])  # rows 0 and 1 share their first two pages (32 tokens)
    # row 0: would write to a shared page; row 2: not ascending; row 3: past the end
    x.compact([16, 30, 40, 10], [[1, 2], [1, -1], [3, 3], [0, 8]], [2, 1, 2, 2])
    assert int(x.cache.status) == q_.KV_SHARED | q_.KV_BAD_INDEX
    # ending on the page border, or keeping in place, needs no page of its own
    x.compact([16, 32, -1, -2], [[-1, -1]] * 4, [0, 0, 0, 0])
    # a count past keep's width, a position past the length
    x.compact([0, 33, 0, 0], [[0, 1]] * 4, [3, 0, -1, 0])


@pytest.mark.parametrize("pages", [1, 8191, 8192, 8193, 40000])
def test_free_pages_are_found_lowest_first(pages):
    """The scan over many pages: free ones only at its far ends."""
    t = torch()
    say("kv scan", pages)
    k = t.zeros(1, pages, 16, 1, 64, dtype=t.float16, device="cuda")
    refs = np.ones(pages, np.int32)
    free = sorted({0, pages // 3, max(pages - 2, 0), pages - 1, min(8192, pages - 1)})
    refs[free] = 0
    c = q_.KvCache(k, k.clone(), _dev(np.full((3, 4), -1)), _dev([0, 0, 0]), _dev(refs))
    n = len(free)
    pos = q_.kv_reserve(c, _cu([16 * (n // 2), 0, 16 * (n - n // 2)]))
    assert [p for p in c.tables.flatten().tolist() if p >= 0] == free
    assert pos.tolist() == [0, 0, 0] and int(c.status) == 0 and bool((c.refs == 1).all())


def test_reserve_many_rows_and_bad_counts():
    t = torch()
    say("kv many rows")
    rows = 3000
    m = Model(7000, 16, rows, 4)
    c = q_.KvCache.empty(1, 7000, 16, 1, 64, rows, 4)
    rng = np.random.default_rng(0)
    for _ in range(3):
        add = rng.integers(0, 20, rows).tolist()
        assert q_.kv_reserve(c, _cu(add)).tolist() == m.reserve(add)
        assert c.tables.tolist() == m.tables and c.refs.tolist() == m.refs and c.lens.tolist() == m.lens
    cu = _cu([3] * rows)
    cu[5] = 2  # descending offsets
    before = c.lens.tolist()
    pos = q_.kv_reserve(c, cu)
    assert pos[4] == -1 and c.lens[4] == before[4] and int(c.status) & q_.KV_BAD_INDEX


def test_keeping_more_tokens_than_a_wave_has_lanes():
    """150 of 200 drafted tokens, and all of them; larger tables than a fork takes in one workgroup."""
    t = torch()
    say("kv long keeps")
    rng = np.random.default_rng(1)
    x = Both(2, 80, 16, 1, 64, 3, 6000, t.float16)
    x.append([37, 0, 100])
    pos = x.append([200, 200, 130])
    keep = [sorted(rng.choice(200, 150, replace=False).tolist()), list(range(150)), [0, 5] + list(range(60, 130)) + [0] * 78]
    x.compact(pos, keep, [150, 150, 72])
    x.fork([2, 0, 0])
    x.append([5, 30, 1])


def test_more_rows_from_fewer_and_back():
    """Forks between caches of different row counts; bf16 pools."""
    t = torch()
    say("kv fork rows")
    x = Both(2, 64, 16, 2, 64, 2, 8, t.bfloat16)
    x.append([37, 50])
    x.fork([0, 1, 0, 1, 1, 0, -1])
    x.append([1, 0, 2, 3, 1, 15, 40])
    x.fork([6, 2])
    x.fork([-1])
    assert sum(x.model.refs) == 0
