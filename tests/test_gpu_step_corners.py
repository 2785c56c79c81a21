"""Corners of the norm, append and sampling calls: more rows than a launch has workgroups for, rows that lie far apart,
rotations of every allowed width, and rows of zeros without an eps."""
import numpy as np
import pytest

from tests import kv8_ref as ref
from tests.gpu_util import say, torch
from tests.test_gpu_append import HALF, Setup, cu_of, ints

pytestmark = pytest.mark.gpu

q = pytest.importorskip("gemm_unpack_bit_amd")

FAR = 1 << 20  # elements between rows: 2100 of them end past 2^31


def apart(rows, shape, dtype, seed):
    """[rows, *shape] whose rows lie FAR apart, and a contiguous copy."""
    t = torch()
    n = int(np.prod(shape))
    x = t.empty(rows * FAR, dtype=dtype, device="cuda").view(rows, FAR)[:, :n]
    x.copy_(t.randn((rows, n), generator=t.Generator(device="cuda").manual_seed(seed), device="cuda"))
    return x.unflatten(1, shape), x.clone().view(rows, *shape)


@pytest.mark.parametrize("rows,dim", [((1 << 22) + 77, 8), ((1 << 20) + 5, 129)])
def test_more_rows_than_workgroups(rows, dim):
    """Rows repeat every 1009, so a few are worked out and all others are the same bits."""
    t = torch()
    say("norm: many rows", rows, dim)
    x = t.randn(1009, dim, generator=t.Generator(device="cuda").manual_seed(1), device="cuda").bfloat16()
    w = t.randn(dim, generator=t.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    many = x.repeat(-(-rows // 1009), 1)[:rows].contiguous()
    want = q.rms_norm(x, w)
    y = q.rms_norm(many, w)
    assert t.equal(y, want.repeat(-(-rows // 1009), 1)[:rows])
    codes, steps = q.rms_norm_q8(many, w)
    wc, ws = q.rms_norm_q8(x, w)
    assert t.equal(codes, wc.repeat(-(-rows // 1009), 1)[:rows]) and t.equal(steps, ws.repeat(-(-rows // 1009))[:rows])


def test_norm_of_rows_that_lie_far_apart():
    t = torch()
    say("norm: far rows")
    far, near = apart(2100, (192,), t.float16, 1)
    out, _ = apart(2100, (192,), t.float16, 2)
    total, _ = apart(2100, (192,), t.float16, 3)
    w = t.ones(192, device="cuda").half()
    y, h = q.rms_norm(far, w, residual=far, out=out, residual_out=total)
    yn, hn = q.rms_norm(near, w, residual=near)
    assert t.equal(y, yn) and t.equal(h, hn)
    assert all(t.equal(a, b) for a, b in zip(q.rms_norm_q8(far, w), q.rms_norm_q8(near, w)))


def test_sample_of_rows_that_lie_far_apart():
    t = torch()
    say("sample: far rows")
    far, near = apart(2100, (5000,), t.float16, 4)
    u = t.rand(2100, generator=t.Generator(device="cuda").manual_seed(5), device="cuda")
    k = (t.arange(2100, device="cuda") % 3 * 40).int()
    p = t.full((2100,), 0.9, device="cuda")
    assert t.equal(q.sample(far, u, top_k=k, top_p=p), q.sample(near, u, top_k=k, top_p=p))


@pytest.mark.parametrize("eight", [False, True])
def test_append_and_read_of_tokens_that_lie_far_apart(eight):
    t = torch()
    say("append, read: far tokens", eight)
    n, kv, heads, dim = 2100, 2, 4, 64
    (k, kn), (v, vn), (x, xn) = (apart(n, (h, dim), t.float16, h + s) for h, s in ((kv, 1), (kv, 7), (heads, 3)))
    freqs = t.tensor([1.0 / (1 + i) for i in range(dim // 2)], device="cuda")
    results = []
    for a in ((k, v, x), (kn, vn, xn)):
        cache = q.KvCache.empty(1, 150, 16, kv, dim, 2, 100, dtype=t.float8_e4m3fn if eight else t.float16)
        cu = cu_of([1000, 1100])
        pos = q.kv_reserve(cache, cu)
        out = q.kv_append(cache, 0, a[0], a[1], cu, pos, q=a[2], freqs=freqs, out=a[2])
        back = (k, v) if a[0] is k else (kn, vn)
        q.kv_read(cache, 0, cu, pos, out=back)
        assert int(cache.status) == 0
        results.append((out, *back))
    assert all(t.equal(a, b) for a, b in zip(*results))


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("eight", [False, True])
@pytest.mark.parametrize("dim", [64, 128])
def test_rotations_of_every_width(dim, eight, dtype):
    t = torch()
    for rot in range(16, dim + 1, 16):
        for inter in (False, True):
            say("append: rotation", dim, eight, dtype, rot, inter)
            s = Setup([3, 30], [20, 5], 16, 3, dim, eight, dtype, seed=rot)
            freqs = (100.0 ** (-2.0 * np.arange(rot // 2) / rot)).astype(np.float32)
            at = np.concatenate([np.arange(3, 23), np.arange(30, 35)])
            k, v, x = s.heads(3), s.heads(3), s.heads(6)
            out = q.kv_append(s.cache, 1, k, v, s.cu, ints(s.pos), q=x, freqs=t.from_numpy(freqs).cuda(), interleaved=inter)
            s.check(1, k, v, at, freqs, inter)
            xs = x.double().cpu().numpy()
            want = ref.rotate(xs, at, freqs, inter)
            tol = np.abs(want) * HALF[dtype] + ref.turn_error(xs, freqs, inter) + 2.0 ** -25
            assert (np.abs(out.double().cpu().numpy() - want) <= tol).all()


@pytest.mark.parametrize("dim", [64, 8200])
def test_rows_of_zeros_without_eps(dim):
    """0 / 0: y is NaN, so there is no step."""
    t = torch()
    say("norm: zeros, eps 0", dim)
    x, w = t.zeros(2, dim, device="cuda").half(), t.ones(dim, device="cuda").half()
    x[1, 0] = 1.0
    y = q.rms_norm(x, w, 0.0)
    assert bool(y[0].isnan().all()) and float(y[1, 0]) == pytest.approx(dim ** 0.5, rel=2.0 ** -11 + 2.0 ** -20)
    codes, steps = q.rms_norm_q8(x, w, 0.0)
    assert bool(steps[0].isnan()) and bool((codes[0] == 0).all()) and int(codes[1, 0]) == 127
