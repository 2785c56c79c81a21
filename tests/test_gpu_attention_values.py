"""GPU tests of attention on scores and values that are not finite, against what
the definition gives: NaN, +inf and -inf each in its place."""
import numpy as np
import pytest

from tests.attn_ref import attend, f64, tolerance
from tests.gpu_util import say, torch
from tests.test_gpu_attention import _cache, _cu, _dt, _gen, _rand, _words

pytestmark = pytest.mark.gpu

q_ = pytest.importorskip("gemm_unpack_bit_amd")


def _kinds(x):
    return np.isnan(x) * 1 + np.isposinf(x) * 2 + np.isneginf(x) * 3


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,causal", [(7, True), (7, False), (300, True), (300, False)])  # narrow and wide kernel
def test_a_scale_of_zero_times_an_infinite_product_is_nan(dtype, D, n, causal):
    """scale 0: all that is seen weighs the same, and 0 * inf is NaN for the queries that see it, whatever its sign."""
    t = torch()
    say("attn_prompt scale 0", dtype, D, n, causal)
    g, dt = _gen(n), _dt(dtype)
    q = t.ones(n, 2, D, dtype=dt, device="cuda")
    v = _rand(g, n, 2, D, dtype=dt)
    for x, at in ((float("-inf"), n // 2), (float("inf"), n // 2), (float("-inf"), 3), (float("inf"), 3)):
        k = _rand(g, n, 2, D, dtype=dt)
        k[at, 0, 3] = x
        out = f64(q_.attn_prompt(q, k, v, _cu([n]), causal=causal, scale=0.0))
        sees = np.arange(n) >= at if causal else np.ones(n, bool)
        assert np.isnan(out[sees, 0]).all()
        assert np.isfinite(out[~sees, 0]).all() and np.isfinite(out[:, 1]).all()


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [5, 60])
def test_a_scale_of_zero_over_the_cache(dtype, n):
    t = torch()
    say("attn_tree scale 0", dtype, n)
    dt, pos = _dt(dtype), 200
    cache, tables = _cache(3, dt, [pos + n], 16, 2, 64, fill=float("nan"))
    q = t.ones(n, 4, 64, dtype=dt, device="cuda")
    p = t.tensor([pos], dtype=t.int32, device="cuda")
    assert np.isfinite(f64(q_.attn_tree(q, cache, 0, _cu([n]), p, scale=0.0))).all()
    at = pos + 2  # a new token: the masked steps
    cache.k[0, int(tables[0, at // 16]), at % 16, 1, 0] = float("-inf")
    out = f64(q_.attn_tree(q, cache, 0, _cu([n]), p, scale=0.0))
    assert np.isfinite(out[:2]).all() and np.isfinite(out[:, :2]).all() and np.isnan(out[2:, 2:]).all()
    at = 9  # a cached one: the others
    cache.k[0, int(tables[0, at // 16]), at % 16, 0, 0] = float("-inf")
    assert np.isnan(f64(q_.attn_tree(q, cache, 0, _cu([n]), p, scale=0.0))[:, :2]).all()


def _check_kinds(out, q, k, v, seen_of, group, scale, what):
    o, qd, kd, vd = f64(out), f64(q), f64(k), f64(v)
    for i in range(q.shape[0]):
        for h in range(q.shape[1]):
            with np.errstate(all="ignore"):
                want = attend(qd[i, h], kd[:, h // group], vd[:, h // group], seen_of(i), scale)[0]
            bad = _kinds(want) != _kinds(o[i, h])
            assert not bad.any(), f"{what}: query {i} head {h}: {o[i, h][bad][:4]} for {want[bad][:4]}"


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,m", [(6, 6), (6, 300), (200, 200), (60, 2500)])  # narrow, wide, wide with split keys
@pytest.mark.parametrize("causal", [True, False])
def test_infinities_and_nan_each_in_their_place(dtype, D, n, m, causal):
    """Values of +inf, -inf and NaN show in the queries that see them, in their column and with their sign; +inf and -inf
    together are NaN; keys of NaN, and scores of +inf, make every column NaN."""
    say("attn_prompt kinds", dtype, D, n, m, causal)
    rng, g, dt = np.random.default_rng(n + m), _gen(n + m), _dt(dtype)
    q = _rand(g, n, 2, D, dtype=dt, scale=0.5)
    k, v = _rand(g, m, 1, D, dtype=dt), _rand(g, m, 1, D, dtype=dt)
    inf = float("inf")
    for at, d, x in ((0, 1, inf), (m // 3, 2, -inf), (m // 2, 3, float("nan")), (m - 1, 4, inf), (m // 2, 5, inf), (m - 2, 5, -inf),
                     (m - n // 2, 6, -inf), (m // 4, D - 1, -inf)):
        v[at, 0, d] = x
    seen = lambda i: np.arange(m) <= i + m - n if causal else np.ones(m, bool)  # noqa: E731
    out = q_.attn_prompt(q, k, v, _cu([n]), _cu([m]), causal=causal)
    _check_kinds(out, q, k, v, seen, 2, D ** -0.5, f"values {n} {m}")
    q.abs_()
    for x in (inf, float("nan")):
        k2 = k.clone()
        k2[m - n // 2 - 1, 0, 0] = x
        out = q_.attn_prompt(q, k2, v, _cu([n]), _cu([m]), causal=causal)
        _check_kinds(out, q, k2, v, seen, 2, D ** -0.5, f"key {x} {n} {m}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("heads,n", [(2, 7), (4, 7), (4, 33), (8, 33)])  # narrow (one and two tiles of rows), wide (4 and 8 waves)
def test_trees_with_infinities_and_nan(dtype, D, heads, n):
    say("attn_tree kinds", dtype, D, heads, n)
    rng, dt, pos = np.random.default_rng(n), _dt(dtype), 131
    cache, tables = _cache(n, dt, [pos + n], 16, 1, D, fill=float("nan"))
    at = lambda p: (0, int(tables[0, p // 16]), p % 16, 0)  # noqa: E731
    inf = float("inf")
    for p, d, x in ((0, 1, inf), (60, 2, -inf), (130, 3, float("nan")), (pos, 4, -inf), (pos + 2, 5, inf), (pos + 3, 5, -inf),
                    (pos + n - 1, 6, float("nan")), (pos + 1, D - 1, inf)):
        cache.v[at(p)][d] = x
    bits = [sorted(rng.choice(n, rng.integers(0, n), replace=False).tolist()) for _ in range(n)]
    q = _rand(_gen(n), n, heads, D, dtype=dt, scale=0.5)
    t = torch()
    out = q_.attn_tree(q, cache, 0, _cu([n]), t.tensor([pos], dtype=t.int32, device="cuda"), _words(bits, 1))
    k = t.stack([cache.k[at(p)] for p in range(pos + n)])[:, None]
    v = t.stack([cache.v[at(p)] for p in range(pos + n)])[:, None]

    def seen(i):
        s = np.arange(pos + n) < pos
        s[[pos + j for j in bits[i]]] = True
        return s

    _check_kinds(out, q, k, v, seen, heads, D ** -0.5, f"tree {n}")


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("n", [4, 150])
def test_scores_of_minus_infinity_weigh_nothing(dtype, n):
    """A seen key whose score is -inf has no weight; a query all of whose scores are has output 0, like one without keys."""
    t = torch()
    say("attn_prompt scores of -inf", dtype, n)
    g, dt = _gen(n), _dt(dtype)
    q, v = t.ones(n, 2, 64, dtype=dt, device="cuda"), _rand(g, n, 2, 64, dtype=dt)
    k = _rand(g, n, 2, 64, dtype=dt)
    k[:n // 2, :, 9] = float("-inf")
    out = f64(q_.attn_prompt(q, k, v, _cu([n])))
    assert (out[:n // 2] == 0).all()
    kd, vd = f64(k), f64(v)
    for i in range(n // 2, n):
        want = attend(np.ones(64), kd[n // 2:i + 1, 1], vd[n // 2:i + 1, 1], np.ones(i + 1 - n // 2, bool), 0.125)[0]
        assert np.abs(out[i, 1] - want).max() < 2.0 ** -6 * np.abs(vd).max()  # (rounding is tested elsewhere)


LARGE = [("f16", 300.0), ("f16", 1500.0), ("f16", 3000.0), ("f16", 5000.0), ("f16", 12000.0), ("bf16", 1e3), ("bf16", 1e5), ("bf16", 1e9),
         ("bf16", 1e15)]


def _check_largest(out, q, k, v, seen_of, group, what):
    """Where a query's largest score is far above the others, its output is that key's value."""
    o, qd, kd, vd = f64(out), f64(q), f64(k), f64(v)
    checked = 0
    for i in range(q.shape[0]):
        seen = np.flatnonzero(seen_of(i))
        for h in range(q.shape[1]):
            assert np.isfinite(o[i, h]).all(), f"{what}: query {i} head {h}"
            s = kd[seen, h // group] @ qd[i, h]
            top = seen[s.argmax()]
            # an fp32 sum of D products is off by D 2^-24 sum |q k| at most; 200 is 2^-288 in weight
            off = q.shape[2] ** 0.5 * 2 * 2.0 ** -24 * (np.abs(kd[seen, h // group]) @ np.abs(qd[i, h])).max()
            if len(s) > 1 and (s.max() - np.sort(s)[-2]) * q.shape[2] ** -0.5 < 200 + off:
                continue
            assert np.abs(o[i, h] - vd[top, h // group]).max() <= 2.0 ** -7 * np.abs(vd[top, h // group]).max(), f"{what}: {i} {h}"
            checked += 1
    assert checked > q.shape[0] // 2


@pytest.mark.parametrize("dtype,size", LARGE)
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,m", [(6, 6), (6, 300), (150, 150), (60, 2500)])  # narrow, wide, wide with split keys
def test_large_scores_leave_the_largest(dtype, size, D, n, m):
    """Scores far beyond what 32 bits hold the units of: weights must neither overflow nor vanish."""
    say("attn_prompt large scores", dtype, size, D, n, m)
    g, dt = _gen(n + m), _dt(dtype)
    q, k = _rand(g, n, 2, D, dtype=dt, scale=size), _rand(g, m, 1, D, dtype=dt, scale=size)
    v = _rand(g, m, 1, D, dtype=dt)
    out = q_.attn_prompt(q, k, v, _cu([n]), _cu([m]))
    _check_largest(out, q, k, v, lambda i: np.arange(m) <= i + m - n, 2, f"{size} {n} {m}")


@pytest.mark.parametrize("dtype,size", LARGE)
@pytest.mark.parametrize("heads,n", [(2, 7), (4, 7), (4, 33), (8, 33)])  # narrow (one and two tiles of rows), wide (4 and 8 waves)
def test_large_scores_over_the_cache(dtype, size, heads, n):
    t = torch()
    say("attn_tree large scores", dtype, size, heads, n)
    dt, pos = _dt(dtype), 700
    cache, tables = _cache(n, dt, [pos + n], 16, 1, 64, fill=float("nan"))
    cache.k.mul_(size)
    q = _rand(_gen(n), n, heads, 64, dtype=dt, scale=size)
    out = q_.attn_tree(q, cache, 0, _cu([n]), t.tensor([pos], dtype=t.int32, device="cuda"))
    at = lambda p: (0, int(tables[0, p // 16]), p % 16, 0)  # noqa: E731
    k = t.stack([cache.k[at(p)] for p in range(pos + n)])[:, None]
    v = t.stack([cache.v[at(p)] for p in range(pos + n)])[:, None]
    _check_largest(out, q, k, v, lambda i: np.arange(pos + n) <= pos + i, heads, f"tree {size} {n}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n", [1, 64])  # narrow and wide kernel
@pytest.mark.parametrize("step", [0.0, 5.2, -5.2])
def test_large_bf16_values_do_not_overflow(D, n, step):
    """Values of 1e36, whose sum over the keys 32 bits hold, while later keys' scores go past the earlier ones'."""
    t = torch()
    say("attn_prompt large values", D, n, step)
    m = 256
    q, k = t.zeros(n, 2, D, dtype=t.bfloat16, device="cuda"), t.zeros(m, 1, D, dtype=t.bfloat16, device="cuda")
    q[:, :, 0] = 1
    k[m // 2:, :, 0] = step
    v = t.full((m, 1, D), 1e36, dtype=t.bfloat16, device="cuda")
    v[:, :, 1::2] *= -1
    out = q_.attn_prompt(q, k, v, _cu([n]), _cu([m]), causal=False, scale=1.0)
    want = v[:1].expand(n, 2, D).double()
    assert bool(((out.double() - want).abs() <= 2.0 ** -7 * want.abs()).all())  # (two roundings of 2^-8)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("n,m", [(3, 40), (64, 300)])  # narrow and wide kernel
@pytest.mark.parametrize("which", ["queries and keys", "values"])
def test_subnormal_fp16_inputs_count(D, n, m, which):
    """Elements below 2^-14, the smallest normal number of fp16."""
    t = torch()
    say("attn_prompt subnormal", D, n, m, which)
    g, tiny = _gen(D + n), 2.0 ** -17
    a, b = (tiny, 1.0) if which == "queries and keys" else (1.0, tiny)
    q, k, v = (_rand(g, x, h, D, dtype=t.float16, scale=c) for x, h, c in ((n, 2, a), (m, 1, a), (m, 1, b)))
    assert 0 < float((v if a == 1 else q).abs().max()) < 2.0 ** -14
    scale = 2.0 * D ** -0.5 / a ** 2  # scores of about 2
    out = f64(q_.attn_prompt(q, k, v, _cu([n]), _cu([m]), causal=False, scale=scale))
    qd, kd, vd = f64(q), f64(k), f64(v)
    for i in range(n):
        for h in range(2):
            want, A, reach = attend(qd[i, h], kd[:, 0], vd[:, 0], np.ones(m, bool), scale)
            tol = tolerance(A, reach, m, D, "f16", np.abs(vd).max())
            assert (np.abs(out[i, h] - want) <= tol).all(), (i, h)
            # (taken for 0, they would give the mean of the values, or 0)
            other = vd[:, 0].mean(0) if b == 1 else np.zeros(D)
            assert (np.abs(other - want) > 4 * tol).any(), "the case does not tell"
