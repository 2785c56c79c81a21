"""GPU tests of writing tokens behind the position rotation, into caches of 16 and of 8 bits, and of reading them back,
against the plain forms of tests/kv8_ref.py.  The whole pools are compared: what no token of the call belongs to stays."""
import numpy as np
import pytest

from tests import kv8_ref as ref
from tests.gpu_util import say, torch

pytestmark = pytest.mark.gpu

q = pytest.importorskip("gemm_unpack_bit_amd")

HALF = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}


def ints(v):
    return torch().tensor(v, dtype=torch().int32, device="cuda")


def cu_of(n):
    return ints([0] + np.cumsum(n).tolist())


class Setup:
    """A cache with given row lengths before the new tokens, over shuffled pages, and its pools on the host."""

    def __init__(self, before, new, page, kv, dim, eight, dtype, layers=2, seed=0, spare=3, lost=()):
        t = self.t = torch()
        self.before, self.new, self.page, self.kv, self.dim, self.eight, self.dtype = before, new, page, kv, dim, eight, dtype
        r = self.rng = np.random.default_rng(seed)
        need = [-(-(a + b) // page) for a, b in zip(before, new)]
        width = max(need + [1]) + 1
        order = r.permutation(sum(need) + spare).tolist()
        self.tables, at = [], 0
        for n in need:
            self.tables.append(order[at:at + n] + [-1] * (width - n))
            at += n
        self.pos = [-1 if b in lost else n for b, n in enumerate(before)]
        pages, rows = len(order), len(before)
        shape = (layers, pages, page, kv, dim)
        g = t.Generator(device="cuda").manual_seed(seed)
        if eight:
            codes = [t.randint(0, 256, shape, generator=g, device="cuda", dtype=t.uint8) for _ in range(2)]
            exps = [t.randint(112, 130, (layers, pages, page // 16, kv), generator=g, device="cuda", dtype=t.uint8) for _ in range(2)]
            self.host = [ref.Pool(c.cpu().numpy(), e.cpu().numpy()) for c, e in zip(codes, exps)]
            self.pools = [*codes, *exps]
            self.start = [c.clone() for c in codes]
            k, v = (c.view(t.float8_e4m3fn) for c in codes)
            more = dict(k_exps=exps[0], v_exps=exps[1])
        else:
            k, v = (t.randn(shape, generator=g, device="cuda").to(getattr(t, dtype)) for _ in range(2))
            self.host = [x.double().cpu().numpy().reshape(layers, pages * page, kv, dim) for x in (k, v)]
            more = {}
        self.cache = q.KvCache(k, v, ints(self.tables).view(rows, width), ints(before), ints([1] * pages), **more)
        self.cu = cu_of(new)

    def heads(self, n, extra=0, scale=1.5):
        """[tokens, n, dim], the middle heads of wider rows."""
        x = self.rng.normal(size=(sum(self.new) + extra, n + 3, self.dim)) * scale
        x = self.t.from_numpy(x).to(getattr(self.t, self.dtype)).cuda()
        return x[:, 1:1 + n]

    def check(self, layer, k, v, at, freqs, interleaved):
        """The pools after k and v (device) have been appended to `layer` at the positions `at` (angles)."""
        u = HALF[self.dtype]
        cu = np.concatenate([[0], np.cumsum(self.new)])
        for which, x in ((0, k), (1, v)):
            x = x.double().cpu().numpy()
            f = freqs if which == 0 else freqs[:0]
            with np.errstate(all="ignore"):
                want, err = ref.rotate(x, at, f, interleaved), ref.turn_error(x, f, interleaved)
            host = self.host[which]
            if not self.eight:
                got = (self.cache.k, self.cache.v)[which].double().cpu().numpy().reshape(host.shape)
                tol = np.zeros(host.shape)
                for b, p0 in enumerate(self.pos):
                    for i in range(self.new[b] if p0 >= 0 else 0):
                        place = self.tables[b][(p0 + i) // self.page] * self.page + (p0 + i) % self.page
                        w = host[layer, place] = want[cu[b] + i]
                        tol[layer, place] = np.abs(w) * u + err[cu[b] + i] + 2.0 ** -25 if len(f) else 0.0
                assert (np.abs(got - host) <= tol).all()
                continue
            got_e = self.pools[2 + which].cpu().numpy().astype(np.int64).reshape(host.e.shape)
            got = ref.values(self.pools[which].cpu().numpy(), self.pools[2 + which].cpu().numpy()).reshape(host.v.shape)
            raw, slack = host.v.copy(), np.zeros(host.v.shape)  # before the new tokens' rounding
            for b, p0 in enumerate(self.pos):
                if p0 < 0 or not self.new[b]:
                    continue
                new, bound = want[cu[b]:cu[b + 1]], err[cu[b]:cu[b + 1]]
                for i, (place, exact) in enumerate(host.append(layer, self.tables[b], p0, new)):
                    raw[layer, place], slack[layer, place] = exact, bound[i] + 1e-300
            old = slack == 0
            # places of the last block behind the row's end: their codes stay, whatever its exponent is now
            behind = np.zeros(host.v.shape[:2], bool)
            for b, p0 in enumerate(self.pos):
                end = p0 + self.new[b]
                if p0 >= 0 and self.new[b]:
                    behind[layer, [host.place(self.tables[b], p) for p in range(end, -(-end // 16) * 16)]] = True
            stay = (self.pools[which] == self.start[which]).cpu().numpy().reshape(host.v.shape)
            assert stay[behind].all()
            # a largest value that lies within the rotation's error of 448 * 2^e may take either exponent
            differ = got_e != host.e
            assert differ.mean() <= (0.01 if len(f) else 0.0)
            assert (np.abs(got_e - host.e) <= 1).all()
            fine = ~np.repeat(differ, 16, axis=1)[..., None] & np.ones(old.shape, bool)
            old &= ~behind[..., None, None]
            assert np.array_equal(got[fine & old], host.v[fine & old], equal_nan=True)
            new = fine & (slack != 0)
            assert np.array_equal(np.isnan(got[new]), np.isnan(raw[new]))
            ok = ~np.isnan(raw[new])
            e = np.repeat(host.e, 16, axis=1)[..., None] + np.zeros(old.shape, np.int64)
            x1, g1 = raw[new][ok], got[new][ok]
            half = ref.step(np.maximum(np.abs(x1), np.abs(g1)), e[new][ok]) / 2
            assert (np.abs(g1 - x1) <= half + slack[new][ok]).all()
            if not len(f):  # nothing before the rounding: the nearest code
                assert np.array_equal(g1, host.v[new][ok])


CASES = [  # before, new
    ([0], [1]), ([15, 16, 17, 31], [1, 1, 1, 1]), ([3, 0, 40], [16, 0, 33]), ([0, 5, 0], [100, 3, 1]),
    ([63, 7, 129, 0, 12], [2, 64, 1, 0, 50]), ([1] * 70, [1] * 70),
]


@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("kv,heads,dim,page", [(1, 4, 64, 16), (8, 32, 128, 16), (3, 0, 128, 64), (2, 20, 64, 32), (5, 7, 128, 256)])
@pytest.mark.parametrize("case", range(len(CASES)))
def test_append(case, kv, heads, dim, page, dtype, eight):
    t = torch()
    before, new = CASES[case]
    if page > 32:
        before, new = before[:9], new[:9]
    for n, (rot, inter, own_at) in enumerate([(dim, False, False), (dim, True, True), (16, False, True), (dim // 2, True, False), (0, False, False)]):
        s = Setup(before, new, page, kv, dim, eight, dtype, seed=n)
        say("append", case, kv, heads, dim, page, dtype, eight, rot, inter)
        freqs = (10000.0 ** (-2.0 * np.arange(rot // 2) / max(rot, 1))).astype(np.float32)
        at = np.concatenate([np.arange(a, a + b) for a, b in zip(before, new)])
        if own_at:
            at = s.rng.integers(0, 1 << 20, len(at))
        k, v, x = s.heads(kv), s.heads(kv), s.heads(heads) if heads else None
        out = q.kv_append(s.cache, 1, k, v, s.cu, ints(s.pos), q=x, freqs=t.from_numpy(freqs).cuda() if rot else None,
                          at=ints(at.tolist()) if own_at and rot else None, interleaved=inter)
        s.check(1, k, v, at, freqs, inter)
        if heads:
            xs = x.double().cpu().numpy()
            want = ref.rotate(xs, at, freqs, inter)
            tol = np.abs(want) * HALF[dtype] + ref.turn_error(xs, freqs, inter) + 2.0 ** -25 if rot else 0.0
            assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()
        else:
            assert out is None


@pytest.mark.parametrize("eight", [False, True])
def test_rows_without_a_place_and_tokens_of_no_row(eight):
    """Rows at -1, tokens behind the last row and positions without a page: nothing of theirs is written, in the result for
    the queries neither."""
    t = torch()
    s = Setup([5, 20, 3], [4, 7, 2], 16, 2, 64, eight, "float16", lost=(1,))
    say("append: skipped rows", eight)
    k, v, x = s.heads(2, extra=6), s.heads(2, extra=6), s.heads(4, extra=6)
    freqs = np.float32(1.0) / (1 + np.arange(32, dtype=np.float32))
    out = t.full(x.shape, 7.0, dtype=x.dtype, device="cuda")
    at = np.concatenate([np.arange(5, 9), np.zeros(7), np.arange(3, 5), np.zeros(6)]).astype(int)
    q.kv_append(s.cache, 0, k, v, s.cu, ints(s.pos), q=x, freqs=t.from_numpy(freqs).cuda(), out=out)
    s.check(0, k, v, at, freqs, False)
    assert bool((out[4:11] == 7).all()) and bool((out[13:] == 7).all()) and bool((out[:4] != 7).any())
    # a page that the row has not: the queries turn, keys and values go nowhere
    s = Setup([14], [4], 16, 2, 64, eight, "float16")
    s.cache.tables[0, 1] = -1
    k, v = s.heads(2), s.heads(2)
    q.kv_append(s.cache, 0, k, v, s.cu, ints(s.pos))
    s.new = [2]
    s.check(0, k[:2], v[:2], np.arange(14, 16), freqs[:0], False)
    # (numbers outside the pool count as no page)
    s.cache.tables[0, :] = 10 ** 6
    after = [a.clone() for a in ((s.cache.k, s.cache.v) if not eight else s.pools)]
    q.kv_append(s.cache, 0, k, v, s.cu, ints(s.pos))
    assert all(t.equal(a.view(t.uint8), b.view(t.uint8)) for a, b in zip(after, (s.cache.k, s.cache.v) if not eight else s.pools))


def test_values_that_are_not_finite_and_exponents_that_grow():
    t = torch()
    s = Setup([0, 10], [20, 3], 16, 2, 128, True, "bfloat16", seed=4)
    say("append8: infinities, NaN, zeros, large and small values")
    k, v = s.heads(2), s.heads(2)
    k[3, 0, 5], k[3, 1, 6], v[4, 0, 7] = float("inf"), float("nan"), -float("inf")
    k[16:20] = 0                        # a block of zeros: the least exponent
    v[16:20] = 3e-30                    # less than it can hold
    v[0:16, 1] = 3e38
    k[20:] *= 1e4                       # codes of the ten tokens before move down by many steps
    v[20:, 1] = float("nan")            # no finite value: what was there stays
    q.kv_append(s.cache, 1, k, v, s.cu, ints(s.pos))
    s.check(1, k, v, np.zeros(23), np.zeros(0, np.float32), False)
    assert int(s.pools[2].view(2, -1, 2)[1, s.tables[0][1], 0]) == 63


def test_the_same_tokens_twice_and_token_by_token():
    """Writing a row again leaves it as it is; token by token gives the same exponents as at once, and values that differ
    by the codes that became subnormal in between only."""
    t = torch()
    say("append8: twice, token by token")
    s = Setup([6], [40], 16, 4, 64, True, "float16", seed=8)
    k, v = s.heads(4), s.heads(4)
    start = [a.clone() for a in s.pools]
    q.kv_append(s.cache, 0, k, v, s.cu, ints(s.pos))
    once = [a.clone() for a in s.pools]
    q.kv_append(s.cache, 0, k, v, s.cu, ints(s.pos))
    assert all(t.equal(a, b) for a, b in zip(once, s.pools))
    for a, b in zip(s.pools, start):
        a.copy_(b)
    for i in range(40):
        q.kv_append(s.cache, 0, k[i:i + 1], v[i:i + 1], ints([0, 1]), ints([6 + i]))
    assert t.equal(s.pools[2], once[2]) and t.equal(s.pools[3], once[3])
    a, b = (ref.values(x.cpu().numpy(), e.cpu().numpy()) for x, e in ((s.pools[0], s.pools[2]), (once[0], once[2])))
    unit = 2.0 ** (np.repeat(once[2].cpu().numpy(), 16, axis=2).astype(float) - 127 - 9)[..., None]  # of subnormal codes
    assert (np.nan_to_num(np.abs(a - b)) <= unit).all()


@pytest.mark.parametrize("eight", [False, True])
def test_queries_in_place_and_in_a_fused_product(eight):
    t = torch()
    say("append: in place", eight)
    s = Setup([3, 9], [5, 30], 16, 2, 128, eight, "bfloat16", seed=2)
    T, H = 35, 6
    qkv = t.from_numpy(s.rng.normal(size=(T, H + 4, 128))).to(t.bfloat16).cuda()
    x, k, v = qkv[:, :H], qkv[:, H:H + 2], qkv[:, H + 2:]
    f = t.tensor([1.0 / (1 + i) for i in range(64)], device="cuda")
    want = q.kv_append(s.cache, 0, k, v, s.cu, ints(s.pos), q=x, freqs=f)
    keep = k.clone()
    got = q.kv_append(s.cache, 0, k, v, s.cu, ints(s.pos), q=x, freqs=f, out=x)
    assert got is x and t.equal(x, want) and t.equal(k, keep)
    with pytest.raises(q.QgemvError):
        q.kv_append(s.cache, 0, k, v, s.cu, ints(s.pos), q=x, freqs=f, out=qkv[:, 1:H + 1])  # over the queries and keys


def test_far_positions():
    t = torch()
    say("append: far positions")
    s = Setup([0], [6], 16, 1, 64, False, "float16")
    at = np.array([0, 1, 131071, 1000003, 16777217, 100000007])
    freqs = np.float32([1.0, 0.75, 0.1, 3e-5] * 8)
    k, v = s.heads(1), s.heads(1)
    q.kv_append(s.cache, 0, k, v, s.cu, ints([0]), freqs=t.from_numpy(freqs).cuda(), at=ints(at.tolist()))
    s.check(0, k, v, at, freqs, False)


@pytest.mark.parametrize("eight,dtype,dim", [(False, "float16", 64), (False, "bfloat16", 128), (True, "float16", 128), (True, "bfloat16", 64)])
def test_read(eight, dtype, dim):
    t = torch()
    s = Setup([40, 3, 0, 17], [0, 1, 0, 90], 32, 3, dim, eight, dtype, seed=6)
    say("read", eight, dtype, dim)
    ends, start = [40, 4, 0, 107], [5, 0, 0, 30]
    n = [e - b for e, b in zip(ends, start)]
    k, v = q.kv_read(s.cache, 1, cu_of(n), ints(start), tokens=sum(n), dtype=getattr(t, dtype) if eight else None)
    i = 0
    for b in range(4):
        for p in range(start[b], ends[b]):
            place = s.tables[b][p // 32] * 32 + p % 32
            for got, host in ((k, s.host[0]), (v, s.host[1])):
                want = (host.v if eight else host)[1, place]
                assert np.array_equal(got[i].double().cpu().numpy(), want, equal_nan=True)
            i += 1
    # rows at -1, tokens of no row and positions without a page stay as they were
    out = [t.full((sum(n) + 4, 5, dim), 3.0, dtype=k.dtype, device="cuda")[:, 1:4] for _ in range(2)]
    q.kv_read(s.cache, 1, cu_of(n), ints([5, -1, 0, 30]), out=out)
    assert t.equal(out[0][:35].view(t.int16), k[:35].view(t.int16)) and bool((out[1][35:39] == 3).all()) and bool((out[0][sum(n):] == 3).all())
    s.cache.tables[3, 2] = -1  # positions 64 .. 95
    out = [t.full(k.shape, 3.0, dtype=k.dtype, device="cuda") for _ in range(2)]
    q.kv_read(s.cache, 1, cu_of(n), ints(start), out=out)
    assert bool((out[0][39 + 34:39 + 66] == 3).all()) and t.equal(out[1][39 + 66:].view(t.int16), v[39 + 66:].view(t.int16))


def test_append_and_read_in_a_graph():
    t = torch()
    say("append8, read: captured")
    s = Setup([9, 30], [1, 1], 16, 2, 64, True, "float16", seed=3)
    k, v, x = s.heads(2), s.heads(2), s.heads(4)
    f, pos, out = t.tensor([1.0 / (1 + i) for i in range(32)], device="cuda"), ints(s.pos), t.empty(2, 4, 64, device="cuda").half()
    all_, zero = cu_of([10, 31]), ints([0, 0])
    back = [t.empty(41, 2, 64, device="cuda").half() for _ in range(2)]

    def run():
        q.kv_append(s.cache, 1, k, v, s.cu, pos, q=x, freqs=f, out=out)
        q.kv_read(s.cache, 1, all_, zero, out=back)

    run()
    t.cuda.synchronize()
    want = [a.clone() for a in (out, *back)]
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        run()
    for _ in range(3):
        for a in (out, *back):
            a.fill_(1)
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        assert all(t.equal(a.view(t.int16), b.view(t.int16)) for a, b in zip((out, *back), want))
