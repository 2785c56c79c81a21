"""GPU tests of attention on scores and values that are not finite, against what
the definition gives: NaN, +inf and -inf each in its place."""
import numpy as np
import pytest

from tests.attn_ref import attend, f64
from tests.gpu_util import say, torch
from tests.test_gpu_attention import _cache, _cu, _dt, _gen, _rand

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
