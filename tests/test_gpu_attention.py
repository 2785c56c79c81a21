"""GPU parity of the attention calls against attention's definition in 64 bits
(tests/attn_ref.py), at the sizes, masks and values where they can go wrong."""
import numpy as np
import pytest

from tests.attn_ref import attend, check, f64
from tests.gpu_util import say, torch

pytestmark = pytest.mark.gpu

q_ = pytest.importorskip("gemm_unpack_bit_amd")


def _dt(name):
    t = torch()
    return t.float16 if name == "f16" else t.bfloat16


def _rand(gen, *shape, dtype, scale=1.0):
    t = torch()
    return (t.randn(*shape, generator=gen, device="cuda") * scale).to(dtype)


def _gen(seed):
    t = torch()
    g = t.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _cu(lens):
    t = torch()
    return t.tensor(np.concatenate([[0], np.cumsum(lens)]).astype(np.int32), device="cuda")


def _sample(n, most, seed):
    """Indices to check of n: all if few, else the ends, tile edges and random ones."""
    if n <= most:
        return list(range(n))
    rng = np.random.default_rng(seed + n)
    fixed = [0, 1, 15, 16, 17, 31, 32, 33, 63, 64, 127, 128, 129, n // 2, n - 2, n - 1]
    return sorted({i for i in fixed if i < n} | set(rng.integers(0, n, max(most - 16, 4)).tolist()))


def _check_prompt(out, q, k, v, nq, nk, causal, scale, dtype, what, most=40):
    o, qd, kd, vd = f64(out), f64(q), f64(k), f64(v)
    D, group = q.shape[2], q.shape[1] // k.shape[1]
    q0 = k0 = 0
    for b, (n, m) in enumerate(zip(nq, nk)):
        vmax = np.abs(vd[k0:k0 + m][np.isfinite(vd[k0:k0 + m])]).max(initial=0.0)
        for i in _sample(n, most, b):
            seen = np.arange(m) <= i + m - n if causal else np.ones(m, bool)
            for h in sorted({0, group - 1, q.shape[1] // 2, q.shape[1] - 1}):
                want, A, reach = attend(qd[q0 + i, h], kd[k0:k0 + m, h // group], vd[k0:k0 + m, h // group], seen, scale)
                check(o[q0 + i, h], want, A, reach, m, D, dtype, vmax, f"{what} seq {b} query {i} head {h}")
        q0, k0 = q0 + n, k0 + m


PROMPTS = [
    # (nq per sequence, nk per sequence or None)
    ([1], None),
    ([3, 1, 0, 7], None),
    ([64], None), ([65], None), ([127, 129], None),
    ([300, 1, 33, 0, 200], None),
    ([5, 70, 2], [5, 200, 64]),          # continuing earlier keys
    ([40, 9], [17, 0]),                  # queries in front of the first key see nothing
    ([1, 2], [1000, 3001]),              # few queries, many keys: split over workgroups
    ([150, 130], [2500, 1000]),
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv,D", [(4, 1, 128), (8, 8, 64), (6, 2, 64), (3, 3, 128), (16, 1, 128)])
@pytest.mark.parametrize("case", range(len(PROMPTS)))
@pytest.mark.parametrize("causal", [True, False])
def test_prompt(dtype, heads, kv, D, case, causal):
    nq, nk = PROMPTS[case]
    say("attn_prompt", dtype, heads, kv, D, nq, nk, causal)
    g, dt = _gen(case * 7 + heads), _dt(dtype)
    nk_ = nk or nq
    q = _rand(g, sum(nq), heads, D, dtype=dt, scale=2.0)
    k, v = _rand(g, sum(nk_), kv, D, dtype=dt), _rand(g, sum(nk_), kv, D, dtype=dt)
    out = q_.attn_prompt(q, k, v, _cu(nq), _cu(nk) if nk else None, causal=causal)
    _check_prompt(out, q, k, v, nq, nk_, causal, D ** -0.5, dtype, f"{nq} {nk}", most=24)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("scale", [0.0, 0.02, 1.0])
def test_prompt_strides_scale_and_out(dtype, scale):
    """Parts of a fused product's rows, an output inside a wider array, a scale of its own."""
    t = torch()
    say("attn_prompt strides", dtype, scale)
    g, dt = _gen(5), _dt(dtype)
    nq, H, KV, D = [37, 150], 8, 2, 128
    T = sum(nq)
    qkv = _rand(g, T, H + 2 * KV, D, dtype=dt)
    q, k, v = qkv[:, :H], qkv[:, H:H + KV], qkv[:, H + KV:]
    wide = t.full((T, H + 3, D), 7.0, dtype=dt, device="cuda")
    out = q_.attn_prompt(q, k, v, _cu(nq), scale=scale, out=wide[:, 2:2 + H])
    _check_prompt(out, q, k, v, nq, nq, True, scale, dtype, "strided")
    assert bool((wide[:, :2] == 7).all()) and bool((wide[:, 2 + H:] == 7).all())
    # heads outermost
    qh, kh, vh = (x.transpose(0, 1).contiguous().transpose(0, 1) for x in (q, k, v))
    oh = t.empty((H, T, D), dtype=dt, device="cuda").transpose(0, 1)
    q_.attn_prompt(qh, kh, vh, _cu(nq), scale=scale, out=oh)
    assert t.equal(oh, out)
    # keys shared by all heads: stride 0
    k1, v1 = k[:, :1].expand(T, H, D), v[:, :1].expand(T, H, D)
    _check_prompt(q_.attn_prompt(q, k1, v1, _cu(nq), scale=scale), q, k1, v1, nq, nq, True, scale, dtype, "broadcast")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,heads", [(200, 2), (9, 1)])  # the wide and the narrow kernel
def test_prompt_what_masked_keys_hold_does_not_matter(dtype, D, n, heads):
    """NaN, infinities and the type's lowest value in later keys and values, and in the next sequence."""
    t = torch()
    say("attn_prompt odd values", dtype, D, n)
    g, dt = _gen(11), _dt(dtype)
    nq = [n, 2 * n]
    q = _rand(g, 3 * n, heads, D, dtype=dt)
    k, v = _rand(g, 3 * n, heads, D, dtype=dt), _rand(g, 3 * n, heads, D, dtype=dt)
    low = t.finfo(dt).min
    for at, x in ((n - 3, float("nan")), (n - 2, float("inf")), (n - 1, low), (n + n // 2, float("-inf")), (3 * n - 1, float("nan"))):
        k[at, :, ::3] = x
        v[at, :, ::2] = x
    out = q_.attn_prompt(q, k, v, _cu(nq))
    _check_prompt(out[:n], q[:n], k[:n], v[:n], [n], [n], True, D ** -0.5, dtype, "first", most=n if n < 50 else 60)
    # the second sequence up to its first odd key
    m = n // 2
    _check_prompt(out[n:n + m], q[n:n + m], k[n:n + m], v[n:n + m], [m], [m], True, D ** -0.5, dtype, "second")
    # only a value is odd, and the rows that see it have it in that column alone
    k, v = _rand(g, 3 * n, heads, D, dtype=dt), _rand(g, 3 * n, heads, D, dtype=dt)
    v[n // 2, 0, 5], v[n // 2, 0, D - 1] = float("inf"), float("nan")
    out = f64(q_.attn_prompt(q, k, v, _cu(nq)))
    assert np.isfinite(out[:n // 2]).all()
    col = out[n // 2:n, 0]
    assert (col[:, 5] == np.inf).all() and np.isnan(col[:, D - 1]).all()
    rest = [d for d in range(D) if d not in (5, D - 1)]
    assert np.isfinite(col[:, rest]).all() and np.isfinite(out[n:]).all()


def test_prompt_rows_without_keys_are_zero_and_empty_calls():
    t = torch()
    say("attn_prompt empty")
    q = t.ones(20, 4, 64, dtype=t.float16, device="cuda")
    k = t.ones(6, 2, 64, dtype=t.float16, device="cuda")
    out = t.full_like(q, float("nan"))
    q_.attn_prompt(q, k, k, _cu([10, 10]), _cu([6, 0]), out=out)
    assert bool((out[:4] == 0).all()) and bool((out[4:10] == 1).all()) and bool((out[10:] == 0).all())
    out.fill_(float("nan"))
    q_.attn_prompt(q, k[:0], k[:0], _cu([10, 10]), _cu([0, 0]), out=out)
    assert bool((out == 0).all())
    assert q_.attn_prompt(q[:0], k, k, _cu([0]), _cu([6])).shape == (0, 4, 64)
    assert q_.attn_prompt(q[:0], k[:0], k[:0], _cu([])).shape == (0, 4, 64)


# ---------------------------------------------------------------------------
# trees over the paged cache
# ---------------------------------------------------------------------------

def _cache(seed, dt, lens, page, kv, D, layers=1, spare=5, fill=None):
    """A cache whose rows hold lens[b] tokens in shuffled pages; unused places hold `fill`."""
    t = torch()
    rng = np.random.default_rng(seed)
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    order = rng.permutation(pages)
    width = max(need + [1]) + 2
    tables = np.full((len(lens), width), -1, np.int32)
    refs, at = np.zeros(pages, np.int32), 0
    for b, n in enumerate(need):
        tables[b, :n] = order[at:at + n]
        refs[order[at:at + n]] = 1
        at += n
    g = _gen(seed)
    k = _rand(g, layers, pages, page, kv, D, dtype=dt)
    v = _rand(g, layers, pages, page, kv, D, dtype=dt)
    if fill is not None:
        used = np.zeros((pages, page), bool)
        for b, n in enumerate(lens):
            for p in range(n):
                used[tables[b, p // page], p % page] = True
        free = t.from_numpy(~used).cuda()
        k[:, free] = fill
        v[:, free] = fill
    dev = lambda a: t.from_numpy(np.ascontiguousarray(a, dtype=np.int32)).cuda()  # noqa: E731
    return q_.KvCache(k, v, dev(tables), dev(np.array(lens)), dev(refs)), tables


def _gather(pool, table, n, page):
    return np.stack([pool[table[p // page], p % page] for p in range(n)]) if n else pool[:0, 0]


def _words(bits, words):
    """Lists of visible tokens -> int64 words."""
    out = np.zeros((len(bits), words), np.uint64)
    for i, js in enumerate(bits):
        for j in js:
            if j < 64 * words:
                out[i, j // 64] |= np.uint64(1 << (j % 64))
    return torch().from_numpy(out.view(np.int64)).cuda()


def _check_tree(out, q, cache, layer, tables, ns, pos, bits, scale, dtype, what, most=24):
    o, qd = f64(out), f64(q)
    kd, vd = f64(cache.k[layer]), f64(cache.v[layer])
    D, group, page = q.shape[2], q.shape[1] // cache.heads_kv, cache.page_size
    q0 = 0
    for b, n in enumerate(ns):
        m = pos[b] + n if pos[b] >= 0 else 0
        k, v = _gather(kd, tables[b], m, page), _gather(vd, tables[b], m, page)
        vmax = np.abs(v[np.isfinite(v)]).max(initial=0.0)
        for i in _sample(n, most, b):
            seen = np.arange(m) < pos[b]
            if m:
                js = range(i + 1) if bits is None else [j for j in bits[q0 + i] if j < n]
                seen[[pos[b] + j for j in js]] = True
            for h in sorted({0, group - 1, q.shape[1] - 1}):
                want, A, reach = attend(qd[q0 + i, h], k[:, h // group], v[:, h // group], seen, scale)
                check(o[q0 + i, h], want, A, reach, m, D, dtype, vmax, f"{what} row {b} token {i} head {h}")
        q0 += n


def _tree(rng, n):
    """Ancestors and self of the nodes of a random tree whose nodes follow their parents."""
    out = []
    for i in range(n):
        p = int(rng.integers(-1, i)) if i else -1
        out.append((out[p] if p >= 0 else []) + [i])
    return out


TREES = [
    # (new tokens per row, tokens before them)
    ([1], [0]), ([1], [776]), ([1, 1, 1], [5, 300, 15]),
    ([1, 0, 1], [31, 7, 2000]),
    ([4, 2], [100, 1]),
    ([13, 30, 1], [0, 77, 500]),
    ([64], [1000]), ([64, 27, 50], [3000, 0, 129]),
    ([1, 5], [-1, 40]),                       # a row that could not grow
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv,D", [(4, 1, 128), (8, 8, 64), (14, 2, 64), (16, 2, 128)])
@pytest.mark.parametrize("page", [16, 64, 256])
@pytest.mark.parametrize("case", range(len(TREES)))
def test_tree(dtype, heads, kv, D, page, case):
    ns, pos = TREES[case]
    say("attn_tree", dtype, heads, kv, D, page, ns, pos)
    rng, g, dt = np.random.default_rng(case + page), _gen(case), _dt(dtype)
    # places without a token hold NaN: nothing of them may come through
    cache, tables = _cache(case, dt, [max(p, 0) + n if p >= 0 else 9 for p, n in zip(pos, ns)], page, kv, D,
                           layers=2, fill=float("nan"))
    q = _rand(g, sum(ns), heads, D, dtype=dt, scale=2.0)
    p = torch().tensor(pos, dtype=torch().int32, device="cuda")
    out = q_.attn_tree(q, cache, 1, _cu(ns), p)
    _check_tree(out, q, cache, 1, tables, ns, pos, None, D ** -0.5, dtype, f"chain {ns} {pos}")
    bits = [b for n in ns for b in _tree(rng, n)]
    bits[0] = []  # sees no new token
    out = q_.attn_tree(q, cache, 1, _cu(ns), p, _words(bits, 1))
    _check_tree(out, q, cache, 1, tables, ns, pos, bits, D ** -0.5, dtype, f"tree {ns} {pos}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv", [(2, 2), (8, 2)])
def test_tree_of_several_mask_words(dtype, heads, kv):
    """More than 64 new tokens; masks at every offset of the key tiles; nodes that see themselves not, or one alone."""
    rng, dt = np.random.default_rng(3), _dt(dtype)
    for n, pos, words in ((70, 31, 2), (150, 90, 3), (130, 64, 2)):
        say("attn_tree words", dtype, heads, n, pos, words)
        cache, tables = _cache(n, dt, [pos + n, 5 + 3], 32, kv, 128, fill=float("inf"))
        bits = [sorted(rng.choice(n, rng.integers(0, n), replace=False).tolist()) for _ in range(n)]
        bits += [[0], [1, 2], []]
        q = _rand(_gen(n), n + 3, heads, 128, dtype=dt)
        p = torch().tensor([pos, 5], dtype=torch().int32, device="cuda")
        out = q_.attn_tree(q, cache, 0, _cu([n, 3]), p, _words(bits, words))
        bits = [[j for j in b if j < 64 * words] for b in bits]
        _check_tree(out, q, cache, 0, tables, [n, 3], [pos, 5], bits, 128 ** -0.5, dtype, f"words {n}", most=40)


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [6, 40])
def test_tree_rows_without_keys_and_odd_values_of_unseen_nodes(dtype, n):
    """pos 0 and an empty mask: 0.  A node with NaN or infinite keys and values shows in the nodes that see it alone."""
    t = torch()
    say("attn_tree odd values", dtype, n)
    dt, D, heads, kv, pos = _dt(dtype), 64, 8, 2, [0, 21]
    cache, tables = _cache(1, dt, [n, 21 + n], 16, kv, D)
    for b in (0, 1):
        for j, x in ((2, float("nan")), (3, float("inf")), (n - 1, float("-inf"))):
            p = pos[b] + j
            cache.k[0, int(tables[b, p // 16]), p % 16, :, 1] = x
            cache.v[0, int(tables[b, p // 16]), p % 16, :, 7] = x
    bits = [[], [1], [1, 2], [0, 3], [0, 1, 4]] + [[0, 1, j] for j in range(5, n)]
    q = _rand(_gen(2), 2 * n, heads, D, dtype=dt)
    p = t.tensor(pos, dtype=t.int32, device="cuda")
    out = q_.attn_tree(q, cache, 0, _cu([n, n]), p, _words(bits * 2, 1))
    o = f64(out)
    assert (o[0] == 0).all()
    odd = [2, 3, n - 1]
    ok = [i for i in range(n) if i not in odd]
    assert np.isfinite(o[ok]).all() and np.isfinite(o[[n + i for i in ok]]).all()
    assert np.isnan(o[[2, n + 2]]).all(-1).all()  # a NaN score: every column
    for b in (0, 1):
        sub = [bits[i] if i in ok else [0] for i in range(n)]
        keep = out.clone()
        for i in odd:
            keep[b * n + i] = q_.attn_tree(q, cache, 0, _cu([n, n]), p, _words(sub * 2, 1))[b * n + i]
        out2 = keep[b * n:(b + 1) * n]
        one, tab = cache, tables[b:b + 1]
        _check_tree(out2, q[b * n:(b + 1) * n], one, 0, tab, [n], [pos[b]], sub, D ** -0.5, dtype, f"odd row {b}", most=n)


@pytest.mark.parametrize("heads,kv,D,ns,pos", [
    (8, 1, 128, [1], [40000]), (64, 8, 128, [1] * 32, [(97 * i * i) % 4001 for i in range(32)]), (32, 8, 128, [1] * 5, [20000, 3, 700, 9000, 64]), (8, 2, 64, [50, 3], [17000, 200]),
])
def test_tree_long_rows(heads, kv, D, ns, pos):
    """Rows of very different lengths: the split of long ones and the join of their parts."""
    say("attn_tree long", heads, kv, D, ns, pos)
    dt = _dt("f16")
    cache, tables = _cache(9, dt, [p + n for p, n in zip(pos, ns)], 64, kv, D, fill=float("nan"))
    q = _rand(_gen(9), sum(ns), heads, D, dtype=dt, scale=3.0)
    p = torch().tensor(pos, dtype=torch().int32, device="cuda")
    out = q_.attn_tree(q, cache, 0, _cu(ns), p)
    _check_tree(out, q, cache, 0, tables, ns, pos, None, D ** -0.5, "f16", "long", most=6)
    assert torch().equal(out, q_.attn_tree(q, cache, 0, _cu(ns), p)), "not deterministic"


def test_tree_many_rows():
    """More rows than a wave has lanes."""
    say("attn_tree many rows")
    rng = np.random.default_rng(4)
    pos = rng.integers(0, 200, 150).tolist()
    ns = [1 if i % 7 else 0 for i in range(150)]
    cache, tables = _cache(4, _dt("f16"), [p + n for p, n in zip(pos, ns)], 16, 2, 64)
    q = _rand(_gen(4), sum(ns), 4, 64, dtype=_dt("f16"))
    p = torch().tensor(pos, dtype=torch().int32, device="cuda")
    out = q_.attn_tree(q, cache, 0, _cu(ns), p)
    _check_tree(out, q, cache, 0, tables, ns, pos, None, 64 ** -0.5, "f16", "many rows")
    out = q_.attn_prompt(q, q[:, :2], q[:, 2:], _cu(ns))
    _check_prompt(out, q, q[:, :2], q[:, 2:], ns, ns, True, 64 ** -0.5, "f16", "many prompts")


@pytest.mark.parametrize("heads,kv,n", [(8, 2, 1), (32, 1, 1), (8, 2, 40)])
def test_what_a_workspace_holds_does_not_matter(heads, kv, n):
    """Parts are joined alike whatever the workspace held: anything on its first use, other shapes' parts later."""
    t = torch()
    say("attn_tree workspace", heads, kv, n)
    dt, pos = _dt("f16"), [9000, 4, 700]
    cache, tables = _cache(21, dt, [p + n for p in pos], 32, kv, 128)
    q, p = _rand(_gen(21), 3 * n, heads, 128, dtype=dt), t.tensor(pos, dtype=t.int32, device="cuda")
    need = q_.attn_tree_workspace_bytes(3 * n, 3, heads, kv, 128)
    ws = t.zeros(need, dtype=t.uint8, device="cuda")
    first = q_.attn_tree(q, cache, 0, _cu([n] * 3), p, ws=ws)
    _check_tree(first, q, cache, 0, tables, [n] * 3, pos, None, 128 ** -0.5, "f16", "workspace", most=4)
    small = _cache(22, dt, [300], 16, kv, 128)[0]
    for fill in (0, 1, 255, "random", "small", "other"):
        if fill == "random":
            ws = t.randint(0, 256, (need,), dtype=t.uint8, device="cuda")
        elif fill == "small":
            ws = t.randint(0, 9, (need // 8,), dtype=t.int64, device="cuda").view(t.uint8)
        elif fill == "other":
            q_.attn_tree(q[:1], small, 0, _cu([1]), p[2:] - 500, ws=ws)
        else:
            ws.fill_(fill)
        for _ in range(3):
            assert t.equal(first, q_.attn_tree(q, cache, 0, _cu([n] * 3), p, ws=ws)), fill


def test_offsets_past_32_bits():
    """A pool of more than 2^32 elements, and packed keys more than 2^31 elements apart."""
    t = torch()
    say("attn_tree far pages")
    layers, pages, page, kv, D = 2, 4300, 256, 16, 128
    cache = q_.KvCache.empty(layers, pages, page, kv, D, 1, 4)
    far = [4299, 4100, 7]
    g = _gen(6)
    for p in far:
        cache.k[1, p].copy_(_rand(g, page, kv, D, dtype=t.float16))
        cache.v[1, p].copy_(_rand(g, page, kv, D, dtype=t.float16))
    cache.tables[0, :3] = t.tensor(far, dtype=t.int32)
    q = _rand(g, 1, 32, D, dtype=t.float16)
    pos = t.tensor([600], dtype=t.int32, device="cuda")
    new = _rand(g, 2, kv, D, dtype=t.float16)
    q_.kv_write(cache, 1, new[:1], new[1:], _cu([1]), pos)
    assert t.equal(cache.k[1, 7, 600 - 512], new[0]) and t.equal(cache.v[1, 7, 600 - 512], new[1])
    out = q_.attn_tree(q, cache, 1, _cu([1]), pos)
    small = q_.KvCache(cache.k[1:, far].contiguous(), cache.v[1:, far].contiguous(),
                       t.tensor([[0, 1, 2, -1]], dtype=t.int32, device="cuda"), cache.lens.clone(),
                       t.zeros(3, dtype=t.int32, device="cuda"))
    assert t.equal(out, q_.attn_tree(q, small, 0, _cu([1]), pos))
    say("attn_prompt far keys")
    heads_apart = (1 << 31) + 64
    big = t.empty(2 * heads_apart, dtype=t.float16, device="cuda")
    k = big.as_strided((300, 2, 64), (64, heads_apart, 1))
    v = big.as_strided((300, 2, 64), (64, heads_apart, 1), 300 * 64)
    k.copy_(_rand(g, 300, 2, 64, dtype=t.float16))
    v.copy_(_rand(g, 300, 2, 64, dtype=t.float16))
    q = _rand(g, 300, 4, 64, dtype=t.float16)
    assert t.equal(q_.attn_prompt(q, k, v, _cu([300])), q_.attn_prompt(q, k.contiguous(), v.contiguous(), _cu([300])))


def test_another_stream_and_a_graph():
    """The calls run on the current stream, and a captured step replays bit for bit."""
    t = torch()
    say("attention on a side stream and in a graph")
    g, dt = _gen(8), _dt("f16")
    H, KV, D, L = 8, 2, 128, 2
    cache = q_.KvCache.empty(L, 40, 16, KV, D, 3, 12)
    # the first step: prompts
    lens = [20, 37, 5]
    cu = _cu(lens)
    pos = q_.kv_reserve(cache, cu)
    kv = [(_rand(g, 62, KV, D, dtype=dt), _rand(g, 62, KV, D, dtype=dt)) for _ in range(L)]
    for layer, (k, v) in enumerate(kv):
        q_.kv_write(cache, layer, k, v, cu, pos)
    state = [x.clone() for x in (cache.tables, cache.lens, cache.refs)]
    q = _rand(g, 9, H, D, dtype=dt)
    k, v = _rand(g, 9, KV, D, dtype=dt), _rand(g, 9, KV, D, dtype=dt)
    cu3 = _cu([3, 3, 3])
    mask = _words([[0], [0, 1], [0, 2]] * 3, 1)
    keep = t.tensor([[0, 2], [0, -1], [0, 1]], dtype=t.int32, device="cuda")
    count = t.tensor([2, 1, 2], dtype=t.int32, device="cuda")
    parents = t.tensor([1, 1, 0], dtype=t.int32, device="cuda")
    p = t.empty(3, dtype=t.int32, device="cuda")
    out = t.empty_like(q)
    pr = t.empty(62, H, D, dtype=dt, device="cuda")
    qp = _rand(g, 62, H, D, dtype=dt)
    nxt = cache.empty_rows()
    need = q_.attn_tree_workspace_bytes(9, 3, H, KV, D), q_.attn_prompt_workspace_bytes(62, 62, 3, H, KV, D)
    ws = t.empty(max(need), dtype=t.uint8, device="cuda")

    def step():
        for a, b in zip((cache.tables, cache.lens, cache.refs), state):
            a.copy_(b)
        q_.attn_prompt(qp, kv[0][0], kv[0][1], cu, out=pr, ws=ws)
        q_.kv_reserve(cache, cu3, out=p)
        q_.kv_write(cache, 1, k, v, cu3, p)
        q_.attn_tree(q, cache, 1, cu3, p, mask, out=out, ws=ws)
        q_.kv_compact(cache, p, keep, count)
        q_.kv_fork(cache, parents, out=nxt)
        return [out, pr, p, cache.refs, nxt.tables, nxt.lens]

    step()
    t.cuda.synchronize()
    eager = [x.clone() for x in step()]
    side = t.cuda.Stream()
    with t.cuda.stream(side):
        for x in (out, pr, p):
            x.fill_(0)
        got = step()
    side.synchronize()
    for a, b in zip(got, eager):
        assert t.equal(a, b)
    graph = t.cuda.CUDAGraph()
    with t.cuda.graph(graph):
        step()
    for rep in range(3):
        out.fill_(float("nan"))
        pr.fill_(float("nan"))
        nxt.tables.fill_(0)
        t.cuda.synchronize()
        say("graph replay", rep)
        graph.replay()
        t.cuda.synchronize()
        for a, b in zip((out, pr, p, cache.refs, nxt.tables, nxt.lens), eager):
            assert t.equal(a, b), rep
