"""GPU tests of the cache of 8 bits: its attention against the definition in 64 bits over the values that it holds,
forks and compaction against a model on the host, and a run of its calls together."""
import numpy as np
import pytest

from tests import attn_ref, kv8_ref as ref
from tests.gpu_util import say, torch

pytestmark = pytest.mark.gpu

q = pytest.importorskip("gemm_unpack_bit_amd")


def ints(v):
    return torch().tensor(v, dtype=torch().int32, device="cuda")


def cu_of(n):
    return ints([0] + np.cumsum(n).tolist())


def pools(layers, pages, page, kv, dim, seed, spread=6):
    """Codes (no NaN) and exponents of values about 1."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    codes, exps = [], []
    for _ in range(2):
        x = t.randn((layers, pages, page, kv, dim), generator=g, device="cuda") * 60
        codes.append(x.clamp(-448, 448).to(t.float8_e4m3fn))
        exps.append(t.randint(127 - 5 - spread, 127 - 5, (layers, pages, page // 16, kv), generator=g, device="cuda", dtype=t.uint8))
    return codes, exps


class Case:
    def __init__(self, lens, new, heads, kv, dim, page, dtype, seed=0, layers=1, layer=0, mask=None):
        t = torch()
        self.lens, self.new, self.layer = lens, new, layer
        need = [-(-(a + b) // page) for a, b in zip(lens, new)]
        order = np.random.default_rng(seed).permutation(sum(need) + 2).tolist()
        width, at, tables = max(need + [1]), 0, []
        for n in need:
            tables.append(order[at:at + n] + [-1] * (width - n))
            at += n
        self.tables, self.page = tables, page
        (k, v), (ke, ve) = pools(layers, len(order), page, kv, dim, seed)
        self.cache = q.KvCache(k, v, ints(tables), ints([a + b for a, b in zip(lens, new)]), ints([1] * len(order)), k_exps=ke, v_exps=ve)
        g = t.Generator(device="cuda").manual_seed(seed + 1)
        self.q = t.randn((sum(new), heads, dim), generator=g, device="cuda").to(getattr(t, dtype))
        self.cu, self.pos, self.mask, self.dtype = cu_of(new), ints(lens), mask, dtype

    def run(self, **more):
        return q.attn_tree(self.q, self.cache, self.layer, self.cu, self.pos, self.mask, **more)

    def values(self):
        c, t = self.cache, torch()
        out = []
        for codes, exps in ((c.k, c.k_exps), (c.v, c.v_exps)):
            x = ref.values(codes.view(t.uint8)[self.layer].cpu().numpy(), exps[self.layer].cpu().numpy())
            out.append(x.reshape(-1, *x.shape[2:]))
        return out

    def check(self, out, what, only=None, scale=None):
        k, v = self.values()
        x = attn_ref.f64(self.q)
        got, (heads, dim), kv = attn_ref.f64(out), self.q.shape[1:], self.cache.heads_kv
        words = None if self.mask is None else self.mask.cpu().numpy().view(np.uint64)
        scale = dim ** -0.5 if scale is None else scale
        i = 0
        for b, (n0, n) in enumerate(zip(self.lens, self.new)):
            places = [self.tables[b][p // self.page] * self.page + p % self.page for p in range(n0 + n)]
            for j in range(n):
                if only is None or i in only:
                    seen = np.zeros(n0 + n, bool)
                    seen[:n0] = True
                    for m in range(n):
                        seen[n0 + m] = m <= j if words is None else bool(int(words[i, m // 64]) >> (m % 64) & 1) if m < 64 * words.shape[1] else False
                    for h in range(heads):
                        kk, vv = k[places, h // (heads // kv)], v[places, h // (heads // kv)]
                        o, A, reach = attn_ref.attend(x[i, h], kk, vv, seen, scale)
                        attn_ref.check(got[i, h], o, A, reach, n0 + n, dim, "f16" if self.dtype == "float16" else "bf16",
                                       np.nanmax(np.abs(vv), initial=0.0), f"{what} row {b} token {j} head {h}")
                i += 1


SHAPES = [(4, 1, 64), (8, 2, 128), (8, 8, 64), (12, 3, 128)]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,kv,dim", SHAPES)
@pytest.mark.parametrize("lens,new,page", [([0], [1], 16), ([777], [1], 16), ([15, 16, 17, 300, 31, 32, 33], [1] * 7, 32),
                                           ([3000, 2, 129], [1, 1, 1], 256), ([50, 0, 7], [3, 2, 0], 64)])
def test_single_tokens(lens, new, page, heads, kv, dim, dtype):
    say("tree8", lens, new, page, heads, kv, dim, dtype)
    c = Case(lens, new, heads, kv, dim, page, dtype, seed=len(lens) + dim, layers=2, layer=1)
    c.check(c.run(), "tree8")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,kv,dim,new", [(16, 1, 128, [40, 9]), (8, 2, 64, [33, 64]), (4, 4, 128, [130, 1]), (32, 4, 128, [5, 6]),
                                              (6, 2, 64, [100, 90])])
def test_many_queries(heads, kv, dim, new, dtype):
    """Rows of more than 32 query rows a key head: the wide kernel, with 4 and with 8 waves; odd lengths around its tiles."""
    for lens in ([0, 0], [1, 63], [64, 200], [1111, 5]):
        say("tree8 wide", heads, kv, dim, new, lens, dtype)
        c = Case(lens, new, heads, kv, dim, 32, dtype, seed=sum(lens))
        c.check(c.run(), "tree8", only={0, 1, new[0] // 2, new[0] - 1, new[0], sum(new) - 1})


@pytest.mark.parametrize("heads,kv,dim,nodes", [(8, 2, 128, 5), (8, 1, 64, 64), (16, 2, 128, 70)])
def test_trees_with_hidden_keys_that_are_not_finite(heads, kv, dim, nodes):
    t = torch()
    r = np.random.default_rng(nodes)
    words = -(-nodes // 64)
    bits = np.zeros((2 * nodes, words), np.uint64)
    for b in range(2):
        for j in range(nodes):
            p = int(r.integers(0, j)) if j else None
            if j % 7 != 3:  # (some nodes see nothing of the tree, themselves included)
                if p is not None:
                    bits[b * nodes + j] = bits[b * nodes + p]
                bits[b * nodes + j, j // 64] |= np.uint64(1) << np.uint64(j % 64)
    mask = t.from_numpy(bits.view(np.int64)).cuda()
    for lens in ([100, 0], [31, 513]):
        say("tree8 masked", heads, kv, dim, nodes, lens)
        c = Case(lens, [nodes, nodes], heads, kv, dim, 16, "float16", seed=3, mask=mask)
        # NaN codes in places that no query sees: behind the row's end, and in a node that only sees itself
        flat = [x.view(t.uint8).view(-1, kv, dim) for x in (c.cache.k, c.cache.v)]
        for b in range(2):
            end = lens[b] + nodes
            for p in range(end, -(-end // 16) * 16):
                for f in flat:
                    f[c.tables[b][p // 16] * 16 + p % 16] = 0x7F
            hidden = lens[b] + 3  # node 3 sees nothing of the tree, and only its children could see it
            others = [j for j in range(nodes) if int(bits[b * nodes + j, 0]) >> 3 & 1]
            if not others:
                for f in flat:
                    f[c.tables[b][hidden // 16] * 16 + hidden % 16] = 0xFF
        out = c.run()
        assert bool(out.isfinite().all())
        c.check(out, "tree8 masked", only=set(range(0, 2 * nodes, 9)) | {3, nodes + 3})


def test_seen_nan_and_values_past_fp16():
    t = torch()
    say("tree8: seen NaN, large exponents")
    c = Case([40, 40], [1, 1], 4, 2, 64, 16, "float16", seed=5)
    c.cache.v.view(t.uint8).view(-1, 2, 64)[c.tables[0][1] * 16 + 2, 1, 9] = 0x7F
    c.cache.v_exps.view(-1, 2)[c.tables[1][0], 0] = 127 + 12  # codes past 16 are past 65504
    out = c.run()
    assert bool(out[0, 2:, 9].isnan().all()) and bool(out[0, :2].isfinite().all()) and int(out[0].isnan().sum()) == 2
    assert not bool(out[1, :2].isfinite().all()) and bool(out[1, 2:].isfinite().all())
    c.q = c.q.bfloat16()
    c.dtype = "bfloat16"
    c.cache.v.view(t.uint8).view(-1, 2, 64)[c.tables[0][1] * 16 + 2, 1, 9] = 0
    c.check(c.run(), "tree8: past fp16, in bf16")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_long_rows_are_split_and_agree_with_16_bits(dtype):
    """The same values in a cache of 16 bits give the same results but for the order of sums."""
    t = torch()
    for new, heads, kv, dim in (([1, 1, 1], 16, 2, 128), ([50, 3, 1], 16, 2, 128), ([1, 1, 1], 8, 8, 64), ([70, 9, 64], 8, 2, 64)):
        lens = [20000, 1, 4500]
        say("tree8 long", new, heads, kv, dim, dtype)
        c = Case(lens, new, heads, kv, dim, 64, dtype, seed=9)
        k, v = (t.from_numpy(x).to(getattr(t, dtype)).cuda().view(c.cache.k.shape) for x in c.values())
        other = q.KvCache(k, v, c.cache.tables, c.cache.lens, c.cache.refs)
        want = q.attn_tree(c.q, other, 0, c.cu, c.pos)
        got = c.run()
        # both round the weights and the output (half a step each), and sum in another order
        vmax, u = float(v.abs().max()), 2.0 ** -11 if dtype == "float16" else 2.0 ** -8
        assert bool(((got.double() - want.double()).abs() <= (4 * u + 20000 * 2.0 ** -23) * vmax).all())
        assert t.equal(got, c.run())
        c.check(got, "tree8 long", only={sum(new[:2]), sum(new) - 1})


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("heads,kv,dim", [(8, 2, 64), (40, 2, 128)])
def test_many_long_rows_on_the_same_pages(heads, kv, dim, dtype):
    """So many keys that a wave takes more than 32 steps of one row in a go; every row reads the same pages."""
    rows, n = 300, 9001
    say("tree8 many long", heads, kv, dim, dtype)
    c = Case([n], [1], heads, kv, dim, 32, dtype, seed=dim)
    c.lens, c.new, c.tables = [n] * rows, [1] * rows, c.tables * rows
    c.cache = q.KvCache(c.cache.k, c.cache.v, ints(c.tables), ints([n + 1] * rows), c.cache.refs, k_exps=c.cache.k_exps,
                        v_exps=c.cache.v_exps)
    c.q = c.q.repeat(rows, 1, 1)
    c.q[1::2] *= -0.5
    c.cu, c.pos = cu_of(c.new), ints(c.lens)
    got = c.run()
    c.check(got, "tree8 many long", only={0, 1, 2, 151, rows - 1})
    # the others: the same queries, with other borders between the parts
    vmax, u = float(max(abs(x).max() for x in c.values())), 2.0 ** -11 if dtype == "float16" else 2.0 ** -8
    for i in (0, 1):
        assert bool(((got[i::2].double() - got[i].double()).abs() <= (4 * u + n * 2.0 ** -23) * vmax).all())


def test_offsets_past_32_bits():
    """The same calls on the last pages of the last layer of 6 GiB pools as on a small cache: the same bits."""
    t = torch()
    say("kv8 offsets past 32 bits")
    kv, heads, dim, page, rows, layers = 8, 32, 128, 256, 3, 3
    lens, more = [300, 1, 511], [1, 40, 2]
    g = t.Generator(device="cuda").manual_seed(3)
    first = [t.randn((sum(lens), kv, dim), generator=g, device="cuda").half() for _ in range(2)]
    new = [t.randn((sum(more), kv, dim), generator=g, device="cuda").half() for _ in range(2)]
    x = t.randn((sum(more), heads, dim), generator=g, device="cuda").half()
    results = []
    for pages in (16, 8192):
        shape = (layers, pages, page, kv, dim)
        k, v = (t.empty(shape, dtype=t.float8_e4m3fn, device="cuda") for _ in range(2))
        ke, ve = (t.empty((layers, pages, page // 16, kv), dtype=t.uint8, device="cuda") for _ in range(2))
        refs = t.ones(pages, dtype=t.int32, device="cuda")
        refs[-16:] = 0  # (only the last ones are free)
        cache = q.KvCache(k, v, t.full((rows, 4), -1, dtype=t.int32, device="cuda"), ints([0] * rows), refs, k_exps=ke, v_exps=ve)
        q.kv_append(cache, 2, *first, cu_of(lens), q.kv_reserve(cache, cu_of(lens)))
        pos = q.kv_reserve(cache, cu_of(more))
        q.kv_append(cache, 2, *new, cu_of(more), pos)
        assert int(cache.status) == 0 and int(cache.tables.max()) < pages and pos.tolist() == lens
        out = [q.attn_tree(x, cache, 2, cu_of(more), pos), q.attn_tree(x[:3], cache, 2, cu_of([1, 1, 1]), pos)]
        out += q.kv_read(cache, 2, cu_of(lens), ints([0] * rows), tokens=sum(lens))
        twin = q.kv_fork(cache, ints([2, 2, 1]))
        q.kv_compact(twin, pos[[2, 2, 1]], ints([[1, 0], [1, 0], [0, 30]]), ints([1, 1, 2]))
        # (token 511 of the first two lies in a full page, which both have, so they are left alone)
        assert int(cache.status) == q.KV_SHARED and twin.lens.tolist() == [513, 513, 3]
        out += q.kv_read(twin, 2, cu_of([513, 513, 3]), ints([0] * rows), tokens=1029)
        results.append(out)
        del k, v, cache, twin
    for a, b in zip(*results):
        assert t.equal(a, b)


def test_rows_at_minus_one_scale_and_strides():
    t = torch()
    say("tree8: rows at -1, scale, strides")
    c = Case([30, 60], [2, 2], 4, 2, 64, 16, "float16", seed=1)
    c.pos = ints([-1, 60])
    assert bool((c.run()[:2] == 0).all())
    c.pos = ints([30, 60])
    wide = t.zeros(4, 9, 64, dtype=t.float16, device="cuda")
    wide[:, 2:6] = c.q
    c.q = wide[:, 2:6]
    out = t.full((4, 5, 64), 7.0, dtype=t.float16, device="cuda")
    c.run(out=out[:, :4], scale=0.5)
    c.check(out[:, :4], "tree8 scaled", scale=0.5)
    assert bool((out[:, 4] == 7).all())
    zero = c.run(scale=0.0)
    c.check(zero, "tree8 scale 0", scale=0.0)


class Both:
    """A cache of 8 bits beside its model: values by kv_append in layers, forks, compaction."""

    def __init__(self, layers, n_pages, page, kv, dim, rows, width, seed=0):
        t = self.t = torch()
        self.cache = q.KvCache.empty(layers, n_pages, page, kv, dim, rows, width, dtype=t.float8_e4m3fn)
        for x in (self.cache.k, self.cache.v):
            x.view(t.uint8).fill_(0x31)
        for x in (self.cache.k_exps, self.cache.v_exps):
            x.fill_(125)
        self.model = attn_ref.Model(n_pages, page, rows, width)
        self.host = [ref.Pool(x.view(t.uint8).cpu().numpy(), e.cpu().numpy())
                     for x, e in ((self.cache.k, self.cache.k_exps), (self.cache.v, self.cache.v_exps))]
        self.rng, self.page = np.random.default_rng(seed), page

    def append(self, add):
        t, c = self.t, self.cache
        want = self.model.reserve(add)
        pos = q.kv_reserve(c, cu_of(add))
        assert pos.tolist() == want
        n = sum(add)
        for layer in range(c.k.shape[0]):
            # sizes that differ from token to token by up to 2^8
            x = self.rng.normal(size=(2, n, c.heads_kv, c.head_dim)) * 2.0 ** self.rng.integers(-4, 5, (2, n, 1, 1))
            k, v = (t.from_numpy(a).half().cuda() for a in x)
            q.kv_append(c, layer, k, v, cu_of(add), pos)
            for host, new in zip(self.host, (k, v)):
                new, at = new.double().cpu().numpy(), 0
                for b, m in enumerate(add):
                    if want[b] >= 0 and m:
                        host.append(layer, self.model.tables[b], want[b], new[at:at + m])
                    at += m
        self.model.write(want, add, list(range(n)))
        self.check(f"append {add}")
        return want

    def fork(self, parents):
        m = self.model
        old = [list(r) for r in m.tables]
        lens = list(m.lens)
        m.fork(parents)
        for i, p in enumerate(parents):
            if p >= 0 and lens[p] % self.page:
                slot = lens[p] // self.page
                if m.tables[i][slot] not in (old[p][slot], -1):
                    for host in self.host:
                        host.copy(old[p][slot], m.tables[i][slot], lens[p] % self.page)
        self.cache = q.kv_fork(self.cache, ints(parents))
        self.check(f"fork {parents}")

    def compact(self, pos, keep, count):
        tables = [list(r) for r in self.model.tables]
        lens = list(self.model.lens)
        self.model.compact(pos, keep, count)
        for b, (p, k, n) in enumerate(zip(pos, keep, count)):
            if p >= 0 and self.model.lens[b] == p + n and lens[b] >= p:
                for host in self.host:
                    host.compact(tables[b], p, list(k[:n]))
        q.kv_compact(self.cache, ints(pos), ints(keep).view(len(pos), -1), ints(count))
        self.check(f"compact {pos} {keep} {count}")

    def check(self, what):
        c, m, t = self.cache, self.model, self.t
        assert c.tables.tolist() == m.tables and c.lens.tolist() == m.lens and c.refs.tolist() == m.refs, what
        assert int(c.status) == m.status, what
        for x, e, host in ((c.k, c.k_exps, self.host[0]), (c.v, c.v_exps, self.host[1])):
            got = ref.values(x.view(t.uint8).cpu().numpy(), e.cpu().numpy()).reshape(host.v.shape)
            ge = e.cpu().numpy().astype(np.int64).reshape(host.e.shape)
            for b, n in enumerate(m.lens):
                places = [m.tables[b][p // self.page] * self.page + p % self.page for p in range(n)]
                if places:
                    blocks = sorted({p // 16 for p in places})
                    assert np.array_equal(ge[:, blocks], host.e[:, blocks]), f"{what}: exponents of row {b}"
                    assert np.array_equal(got[:, places], host.v[:, places], equal_nan=True), f"{what}: values of row {b}"


@pytest.mark.parametrize("page,kv,dim", [(16, 2, 64), (32, 1, 128), (64, 9, 64), (256, 3, 128)])
def test_append_fork_compact(page, kv, dim):
    say("cache of 8 bits: all calls", page, kv, dim)
    b = Both(2, 40, page, kv, dim, 4, 12, seed=page)
    b.append([5, page + 3, 0, 2 * page])
    b.append([1, 1, 1, 1])
    b.fork([1, 1, 3, 0])
    pos = b.append([20, 20, 20, 20])
    # keep: scattered nodes; the first ones in place; all; none
    b.compact(pos, [[0, 3, 4, 9, 17, 19], [0, 1, 2, 0, 0, 0], [1, 2, 3, 4, 5, 6], [0] * 6], [6, 3, 6, 0])
    b.append([3, 0, 40, 1])
    b.fork([0, 0, 2, -1])
    pos = b.append([1, 2, 3, 0])
    b.compact([pos[0], -1, pos[2], 0], [[0], [0], [2], [0]], [1, 0, 1, 0])


def test_compact_of_many_tokens_and_layers():
    say("cache of 8 bits: compaction over many blocks")
    b = Both(5, 30, 32, 4, 128, 2, 14, seed=3)
    b.append([10, 33])
    pos = b.append([200, 150])
    r = np.random.default_rng(0)
    keep = [sorted(r.choice(200, 120, replace=False).tolist()), sorted(r.choice(150, 120, replace=False).tolist())]
    b.compact(pos, keep, [120, 77])
    b.append([7, 60])


def test_compact_refuses_rows_as_16_bits_does():
    say("cache of 8 bits: compaction of bad rows")
    b = Both(1, 20, 16, 2, 64, 3, 8)
    b.append([20, 20, 20])
    b.fork([0, 0, 2])
    b.compact([4, 17, 30], [[0, 2], [1, 0], [0, 1]], [2, 2, 1])  # writes to a shared page; not ascending; past the end


def test_fork_moves_exponents_of_many_heads_and_rows():
    say("cache of 8 bits: wide fork")
    b = Both(3, 80, 64, 20, 64, 30, 3, seed=5)
    b.append([(7 * i) % 90 for i in range(30)])
    b.fork([i // 3 for i in range(30)])


def test_a_run_of_calls_agrees_with_plain_attention():
    """Prompts, a fork, drafted trees, compaction and decode steps, with the attention of each step checked against the
    values that the cache then holds."""
    t = torch()
    say("cache of 8 bits: a serving loop")
    rows, heads, kv, dim = 3, 8, 2, 64
    c = q.KvCache.empty(2, 60, 16, kv, dim, rows, 16, dtype=t.float8_e4m3fn)
    g = t.Generator(device="cuda").manual_seed(1)
    freqs = t.tensor([100.0 ** (-i / 32) for i in range(32)], device="cuda")

    def step(c, add, mask=None, at=None):
        n = sum(add)
        make = lambda h: t.randn((n, h, dim), generator=g, device="cuda").half()  # noqa: E731
        x, k, v = make(heads), make(kv), make(kv)
        cu = cu_of(add)
        pos = q.kv_reserve(c, cu)
        for layer in range(2):
            turned = q.kv_append(c, layer, k, v, cu, pos, q=x, freqs=freqs, at=at)
            out = q.attn_tree(turned, c, layer, cu, pos, mask)
            s = Case.__new__(Case)
            s.lens, s.new, s.layer, s.tables, s.page = pos.tolist(), add, layer, c.tables.tolist(), 16
            s.cache, s.q, s.cu, s.pos, s.mask, s.dtype = c, turned, cu, pos, mask, "float16"
            s.check(out, "loop")
        return pos

    step(c, [40, 3, 17])
    step(c, [1, 1, 1])
    c = q.kv_fork(c, ints([0, 0, 2]))
    bits = [[1 | (1 << j)] for _ in range(3) for j in range(6)]
    pos = step(c, [6, 6, 6], t.tensor(bits, device="cuda"), ints([7 + (j > 0) for _ in range(3) for j in range(6)]))
    q.kv_compact(c, pos, ints([[0, 4], [0, 0], [0, 5]]), ints([2, 1, 2]))
    step(c, [1, 1, 1])
    assert int(c.status) == 0 and c.lens.tolist() == [44, 43, 21]
    # the cached tokens as a prompt's earlier keys: the same as over the cache
    lens = c.lens.tolist()
    k, v = q.kv_read(c, 1, cu_of(lens), ints([0] * 3), tokens=sum(lens))
    x = t.randn((6, heads, dim), generator=g, device="cuda").half()
    packed = q.attn_prompt(x, k, v, cu_of([2, 2, 2]), cu_of(lens))
    over = q.attn_tree(x, c, 1, cu_of([2, 2, 2]), ints([n - 2 for n in lens]))
    # (each rounds its weights and its output)
    assert bool(((packed - over).abs().float() <= 4 * 2.0 ** -11 * float(v.abs().max())).all())


def test_trees_in_a_graph_and_on_another_stream():
    t = torch()
    say("tree8: captured")
    c = Case([300, 4000], [1, 1], 16, 2, 128, 16, "float16", seed=2)
    w = Case([300, 400], [20, 30], 16, 2, 128, 16, "bfloat16", seed=2)
    outs = [t.empty_like(c.q), t.empty_like(w.q)]
    ws = [t.empty(q.attn_tree_workspace_bytes(x.q.shape[0], 2, 16, 2, 128), dtype=t.uint8, device="cuda") for x in (c, w)]

    def run():
        c.run(out=outs[0], ws=ws[0])
        w.run(out=outs[1], ws=ws[1])

    run()
    t.cuda.synchronize()
    want = [o.clone() for o in outs]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        run()
    t.cuda.synchronize()
    assert all(t.equal(a, b) for a, b in zip(outs, want))
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        run()
    for _ in range(3):
        for o in outs:
            o.fill_(0)
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        assert all(t.equal(a, b) for a, b in zip(outs, want))
