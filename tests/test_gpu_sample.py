"""GPU tests of sampling against its definition in 64 bits: the token has to be the same."""
import numpy as np
import pytest

from tests.gpu_util import say, torch

pytestmark = pytest.mark.gpu

q = pytest.importorskip("gemm_unpack_bit_amd")


def choose(x, u, t=1.0, k=0, p=1.0, low=0.0):
    """One row: x float64 logits (NaN as -infinity)."""
    x = np.where(np.isnan(x), -np.inf, x)
    top = x.max()
    if top == -np.inf:
        return -1
    if not t > 0:
        return int(np.argmax(x))
    with np.errstate(all="ignore"):
        w = np.where(x == top, 1.0, np.where(x == -np.inf, 0.0, np.exp((x - top) / t)))
    order = np.argsort(-x, kind="stable")
    order = order[x[order] > -np.inf]
    if 0 < k < order.size:
        order = order[:k]
    if p < 1:
        sums = np.cumsum(w[order])
        order = order[:1 + int(np.searchsorted(sums[:-1], max(p, 0.0) * sums[-1], side="left"))]
    if low > 0:
        order = order[w[order] >= min(low, 1.0)]
    order = np.sort(order)
    sums = np.cumsum(w[order])
    return int(order[min(int(np.searchsorted(sums, u * sums[-1], side="right")), order.size - 1)])


def run(x, u, **settings):
    t = torch()
    d = lambda v, dtype: None if v is None else t.tensor(v, dtype=dtype, device="cuda")  # noqa: E731
    got = q.sample(x, d(u, t.float32), d(settings.get("t"), t.float32), d(settings.get("k"), t.int32),
                   d(settings.get("p"), t.float32), d(settings.get("low"), t.float32))
    return got.tolist()


def check(x, u, what, **settings):
    say("sample", what, tuple(x.shape), x.dtype)
    f32 = lambda v: [float(np.float32(a)) for a in v]  # noqa: E731
    got = run(x, u, **settings)
    rows = x.double().cpu().numpy()
    for r in range(len(rows)):
        mine = {n: (f32(v) if n != "k" else v)[r] for n, v in settings.items()}
        assert got[r] == choose(rows[r], f32(u)[r], **mine), (what, r, u[r], mine)


def logits(rows, vocab, dtype, seed, scale=2.5):
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    return (t.randn((rows, vocab), generator=g, device="cuda") * scale).to(getattr(t, dtype))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16", "float32"])
@pytest.mark.parametrize("rows,vocab", [(1, 1), (5, 2), (3, 63), (17, 1000), (2, 2048), (4, 2049), (33, 9973), (2, 131072), (1, 200001)])
def test_settings(rows, vocab, dtype):
    x = logits(rows, vocab, dtype, vocab)
    r = np.random.default_rng(vocab + rows)
    u = r.random(rows).astype(np.float32).tolist()
    pick = lambda v: r.choice(v, rows).tolist()  # noqa: E731
    check(x, u, "plain")
    check(x, u, "temperature", t=pick([0.0, 0.3, 0.7, 1.0, 2.0]))
    check(x, u, "top_k", t=pick([0.5, 1.0]), k=pick([0, 1, 2, 50, vocab, vocab + 5, 5000]))
    check(x, u, "top_p", t=pick([0.5, 1.0, 3.0]), p=pick([0.0, 0.1, 0.5, 0.9, 0.99, 1.0]))
    check(x, u, "min_p", t=pick([0.5, 1.0]), low=pick([0.0, 0.01, 0.3, 1.0, 2.0]))
    check(x, u, "all", t=pick([0.0, 0.5, 1.0, 3.0]), k=pick([0, 3, 50, 6000]), p=pick([0.3, 0.9, 1.0]), low=pick([0.0, 0.02]))


@pytest.mark.parametrize("dtype", ["float16", "float32"])
def test_many_equal_logits(dtype):
    t = torch()
    n = 30000
    x = t.zeros(6, n, device="cuda", dtype=getattr(t, dtype))
    x[1, 7000:20000] = 1.0            # one step above the rest
    x[2, ::2] = -1.0
    x[3, 5] = 9.0                     # an outlier
    x[4] = -3.0
    x[4, 100] = -1e4                  # all but one in the first bin
    x[5, :] = (t.arange(n, device="cuda") % 7).to(x.dtype)
    u = [0.0, 0.25, 0.5, 0.75, 0.999, 0.3]
    for k in (1, 4096, 4097, 9000, 29999):
        check(x, u, f"equal, top_k {k}", k=[k] * 6)
    for p in (0.0, 0.25, 0.5, 0.75):
        check(x, u, f"equal, top_p {p}", p=[p] * 6)
        check(x, u, f"equal, both {p}", k=[20000] * 6, p=[p] * 6)
    check(x, u, "equal, min_p", low=[1.0] * 6)


def test_close_keys_in_one_bin():
    """A far outlier puts all others into few bins, which are cut by their keys: several levels, in 32 bits."""
    t = torch()
    x = logits(4, 60000, "float32", 9, 1.0)
    x[0, 17] = -1e30
    x[1, 17] = -3e38
    x[2, 17] = 3e38
    x[3, 17], x[3, 18] = -3e38, 3e38
    u = [0.1, 0.9, 0.5, 0.2]
    for k in (1, 10, 4096, 5000, 59000):
        check(x, u, f"outlier, top_k {k}", k=[k] * 4)
    for p in (0.1, 0.9, 0.999):
        check(x, u, f"outlier, top_p {p}", p=[p] * 4)
        check(x, u, f"outlier, both {p}", k=[30000] * 4, p=[p] * 4)


@pytest.mark.parametrize("dtype,min_p", [("float32", 0.0), ("float32", 0.003), ("float16", 0.0)])
def test_every_length_of_the_list(dtype, min_p):
    """Prefixes that end after one, hundreds and thousands of tokens, by count and by weight of these."""
    ks = [1, 2, 63, 64, 65, 255, 256, 257, 300, 511, 512, 513, 1000, 1900, 2031, 2032, 2033, 5000, 40000]
    n = len(ks)
    x = logits(2 * n, 60007, dtype, 41, 2.0)
    u = [(0.37 * i) % 1.0 for i in range(2 * n)]
    check(x, u, "list lengths", k=ks * 2, p=[1.0] * n + [0.93] * n, low=[min_p] * (2 * n))


def test_prefixes_by_weight_alone():
    """... and by weight alone, with min-p above, in and below the bin where they end."""
    ps = [0.001, 0.1, 0.5, 0.9, 0.99, 0.9999]
    x = logits(4 * len(ps), 150001, "float32", 42, 1.5)
    u = [(0.61 * i) % 1.0 for i in range(4 * len(ps))]
    check(x, u, "by weight", p=ps * 4, low=sum(([v] * len(ps) for v in (0.0, 0.5, 0.01, 0.0001)), []), t=[1.0, 0.7] * (2 * len(ps)))


def test_masked_rows():
    t = torch()
    inf = float("inf")
    x = logits(8, 5000, "bfloat16", 4)
    x[0] = -inf                        # nothing is left
    x[1] = float("nan")
    x[2, :4000] = -inf
    x[3, 1:] = -inf
    x[4, 3000], x[4, 3001] = inf, inf  # infinite ones only
    x[5, ::3] = float("nan")
    x[6, 4999] = inf
    x[7] = -inf
    x[7, 4321] = -1e30
    u = [0.5] * 8
    want = dict(t=[1.0] * 8, k=[40] * 8, p=[0.9] * 8, low=[0.001] * 8)
    check(x, u, "masked")
    for drop in want:
        check(x, u, f"masked, without {drop}", **{n: v for n, v in want.items() if n != drop})
    check(x, u, "masked, all", **want)
    check(x, u, "masked, greedy", t=[0.0] * 8)
    assert run(x, u)[:2] == [-1, -1] and run(x, [0.7] * 8)[4] == 3001 and run(x, [0.0] * 8)[4] == 3000


def test_settings_out_of_range():
    inf, nan = float("inf"), float("nan")
    x = logits(6, 3000, "float16", 12)
    u = [0.4] * 6
    check(x, u, "temperature", t=[-1.0, nan, inf, 1e-30, 1e30, 0.0])
    check(x, [-1.0, 0.0, 0.99999994, 0.5, 0.5, 0.5], "u at its ends")
    assert run(x, [2.0, inf, nan, -inf, 0.5, 0.5])[:4] == run(x, [0.99999994, 0.99999994, 0.0, 0.0, 0.5, 0.5])[:4]
    off = run(x, u)
    assert run(x, u, k=[-1, 0, 3000, 2 ** 31 - 1, -2 ** 31, 5000]) == off
    assert run(x, u, p=[1.0, 1.5, nan, inf, 1.0, 2.0]) == off
    assert run(x, u, low=[0.0, -1.0, nan, -inf, 0.0, -0.5]) == off
    first = run(x, u, t=[0.0] * 6)
    assert run(x, u, p=[-1.0, -inf, 0.0, -0.5, 0.0, 0.0]) == first
    assert run(x, u, low=[1.0, 2.0, inf, 1.0, 1.0, 9.0]) == [choose(r, 0.4, low=1.0) for r in x.double().cpu().numpy()]


def test_strided_rows_other_streams_and_graphs():
    t = torch()
    big = logits(7, 4001, "bfloat16", 20)
    x = big[:, 1:3990]  # rows that begin at odd elements
    u = [0.1 * i for i in range(7)]
    check(x, u, "strided", p=[0.9] * 7, k=[300] * 7)
    du, dp, dk = (t.tensor(v, device="cuda") for v in (u, [0.9] * 7, [300] * 7))
    dk = dk.int()
    out, ws = t.empty(7, dtype=t.int32, device="cuda"), t.empty(q.sample_workspace_bytes(7, 3989), dtype=t.uint8, device="cuda")
    ws.fill_(255)
    want = q.sample(x, du, top_p=dp, top_k=dk)
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        assert t.equal(q.sample(x, du, top_p=dp, top_k=dk, out=out, ws=ws), want)
    t.cuda.synchronize()
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        q.sample(x, du, top_p=dp, top_k=dk, out=out, ws=ws)
    for _ in range(3):
        out.fill_(-7)
        ws.fill_(170)
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        assert t.equal(out, want)


def test_graphs_that_share_a_workspace():
    """Two captured calls of different shapes and settings, replayed in turn with eager calls between, all in one
    workspace."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(5)
    ws = t.full((q.sample_workspace_bytes(9, 40000),), 0xA5, dtype=t.uint8, device="cuda")
    calls = []
    for rows, vocab, dtype in ((9, 40000, t.float32), (4, 1003, t.float16)):
        say("sample, shared workspace", rows, vocab)
        x = (t.randn((rows, vocab), generator=g, device="cuda") * 3).to(dtype)
        more = dict(temperature=t.rand(rows, generator=g, device="cuda") + 0.5,
                    top_k=t.randint(0, 60, (rows,), generator=g, device="cuda", dtype=t.int32),
                    top_p=t.rand(rows, generator=g, device="cuda") * 0.5 + 0.5, ws=ws)
        calls.append((x, t.rand(rows, generator=g, device="cuda"), more, t.empty(rows, dtype=t.int32, device="cuda")))
    want = [q.sample(x, u, **more) for x, u, more, _ in calls]
    graphs = []
    for x, u, more, out in calls:
        q.sample(x, u, out=out, **more)
        t.cuda.synchronize()
        graphs.append(t.cuda.CUDAGraph())
        with t.cuda.graph(graphs[-1]):
            q.sample(x, u, out=out, **more)
    for turn in range(3):
        for i in (0, 1, 1, 0):
            calls[i][3].fill_(-7)
            graphs[i].replay()
            x, u, more, out = calls[1 - i]
            assert t.equal(q.sample(x, u, **more), want[1 - i])
            assert t.equal(calls[i][3], want[i])


def test_the_same_call_gives_the_same_tokens():
    t = torch()
    x = logits(64, 50000, "float32", 31)
    u, p = t.rand(64, device="cuda"), t.full((64,), 0.97, device="cuda")
    first = q.sample(x, u, top_p=p)
    for _ in range(5):
        assert t.equal(q.sample(x, u, top_p=p), first)
