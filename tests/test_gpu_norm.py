"""GPU tests of the norm, its 8-bit result and the product that takes it,
against their definitions in 64 bits."""
import numpy as np
import pytest

import synth
from tests.gpu_util import dev, say, torch

pytestmark = pytest.mark.gpu

q = pytest.importorskip("gemm_unpack_bit_amd")

EPS = {"float16": 2.0 ** -11, "bfloat16": 2.0 ** -8}  # half a step, relative
# The factor 1 / sqrt(mean + eps) in 32 bits: a thread's serial sum of dim / 64 squares at most, 6 levels of lanes and 16
# of waves, the division and root, two products: (dim / 64 + 30) roundings of 2^-24.
gamma = lambda dim: (dim / 64 + 30) * 2.0 ** -24  # noqa: E731


def _inputs(rows, dim, dtype, seed, shift=0, pad=0):
    """x, residual and a place for two results, as views of rows `pad` elements longer, `shift` elements in."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(seed)
    make = lambda s: (t.randn((rows, dim + pad + shift), generator=g, device="cuda") * s).to(dtype)[:, shift:shift + dim]  # noqa: E731
    w = (1 + 0.3 * t.randn(dim + shift, generator=g, device="cuda")).to(dtype)[shift:]
    return make(0.8), make(2.0), w, make(0), make(0)


def _exact(x, r, w, eps):
    h = x.double() + (r.double() if r is not None else 0)
    return h, h * w.double() / (h.square().mean(-1, keepdim=True) + eps).sqrt()


def _check(y, want, dtype, dim, extra=0.0):
    name = str(dtype).split(".")[1]
    tol = want.abs() * (EPS[name] + gamma(dim)) * (1 + 2.0 ** -7) + extra + (2.0 ** -25 if name == "float16" else 0)
    assert bool(((y.double() - want).abs() <= tol).all())


SHAPES = [(1, 4096), (1, 1), (3, 7), (70, 64), (5, 8192), (129, 1000), (66, 77), (300, 2048), (2, 33000), (1, 40001), (65, 2056),
          (4097, 128), (90, 16384)]


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_norm(rows, dim, dtype):
    t = torch()
    dt = getattr(t, dtype)
    for layout in ("plain", "strided", "odd"):
        shift, pad = {"plain": (0, 0), "strided": (8, 24), "odd": (1, 2)}[layout]
        x, r, w, y, h = _inputs(rows, dim, dt, 3, shift, pad)
        say("rms_norm", rows, dim, dtype, layout)
        _, want = _exact(x, None, w, 1e-5)
        _check(q.rms_norm(x, w, 1e-5), want, dt, dim)
        _, want = _exact(x, r, w, 1e-5)
        # (the sum in 32 bits is off by half a step of it)
        extra = want.abs() * 2.0 ** -24
        a, b = q.rms_norm(x, w, 1e-5, residual=r, out=y, residual_out=h)
        assert a is y and b is h
        _check(a, want, dt, dim, extra)
        assert t.equal(b, (x.float() + r.float()).to(dt))
        # in place: the norm over x, the sum over the residual, and the other way round
        x2, r2 = x.clone(), r.clone()
        q.rms_norm(x2, w, 1e-5, residual=r2, out=x2, residual_out=r2)
        assert t.equal(x2, a) and t.equal(r2, b)
        x2, r2 = x.clone(), r.clone()
        q.rms_norm(x2, w, 1e-5, residual=r2, out=r2, residual_out=x2)
        assert t.equal(r2, a) and t.equal(x2, b)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("rows,dim", SHAPES)
def test_norm_q8(rows, dim, dtype):
    t = torch()
    dt = getattr(t, dtype)
    for shift, pad in ((0, 0), (1, 3)):
        x, r, w, _, h = _inputs(rows, dim, dt, 5, shift, pad)
        say("rms_norm_q8", rows, dim, dtype, shift)
        _, y = _exact(x, r, w, 1e-6)
        step = y.abs().amax(-1) / 127
        codes, scales, s = q.rms_norm_q8(x, w, 1e-6, residual=r, residual_out=h)
        assert t.equal(s, (x.float() + r.float()).to(dt))
        rel = gamma(dim) + 2.0 ** -22  # (and the sum's, the products' and the division's roundings)
        assert bool(((scales.double() - step).abs() <= step * rel).all())
        # the nearest code, or its neighbour where the quotient is that near to the middle
        off = (codes.double() - y / step[:, None]).abs()
        assert bool((off <= 0.5 + 127 * 2 * rel + 127 * 2.0 ** -23).all())
        plain = q.rms_norm_q8(x, w, 1e-6)
        _, y = _exact(x, None, w, 1e-6)
        off = (plain[0].double() - y / (y.abs().amax(-1) / 127)[:, None]).abs()
        assert len(plain) == 2 and bool((off <= 0.5 + 127 * 2 * rel).all())


@pytest.mark.parametrize("rows,dim", [(500, 4096), (64, 1003), (3, 20000)])
def test_codes_do_not_depend_on_the_weights_power_of_two(rows, dim):
    """Steps far from 1 take the division itself, the others its reciprocal with two corrections: the same codes."""
    t = torch()
    x, r, w, _, _ = _inputs(rows, dim, t.bfloat16, 17)
    say("rms_norm_q8, weights of far powers of two", rows, dim)
    codes, scales, _ = q.rms_norm_q8(x, w, 1e-6, residual=r)
    for e in (-110, -90, 60, 110):  # (all but the smallest magnitudes, whose codes are 0, stay normal numbers)
        c, s, _ = q.rms_norm_q8(x, (w.double() * 2.0 ** e).to(t.bfloat16), 1e-6, residual=r)
        assert t.equal(s.double(), scales.double() * 2.0 ** e) and t.equal(c, codes)


@pytest.mark.parametrize("dim", [64, 8200])
def test_rows_that_are_not_finite_or_zero(dim):
    t = torch()
    say("norm: zero, infinite and NaN rows", dim)
    x = t.randn(5, dim, device="cuda").half()
    x[0] = 0
    x[1, 3], x[2, dim - 1], x[3, 0] = float("inf"), float("nan"), -float("inf")
    w = t.ones(dim, device="cuda").half()
    y = q.rms_norm(x, w)
    assert bool((y[0] == 0).all()) and bool(y[4].isfinite().all())
    assert bool(y[1, 3].isnan()) and bool((y[1, :3] == 0).all()) and bool(y[2].isnan().all()) and bool(y[3, 0].isnan())
    codes, scales = q.rms_norm_q8(x, w)
    assert float(scales[0]) == 0 and bool(scales[1:4].isnan().all()) and float(scales[4]) > 0
    assert bool((codes[:4] == 0).all()) and int(codes[4].abs().max()) == 127


@pytest.mark.parametrize("M,N,K", [(1, 512, 1024), (4, 6144, 4096), (16, 1000, 2176), (13, 17, 128)])
def test_product_of_ready_rows_is_that_of_w4a8(M, N, K):
    t = torch()
    say("w4a8_rows", M, N, K)
    c = synth.uniform_case(91, M, N, K, 4)
    x, wq, s, z = dev(c["x"]), q.pack(dev(c["codes"]), 4), dev(c["scales"]), q.pack_zeros(dev(c["zeros"]), 4)
    ws = t.zeros(q.w4a8_workspace_bytes(M, K), dtype=t.uint8, device="cuda")
    want = q.w4a8(x, wq, s, z, ws)
    x8 = ws[:M * K].view(t.int8).view(M, K)
    step = ws[(M * K + 15) // 16 * 16:][:4 * M].view(t.float32)
    assert t.equal(q.w4a8_rows(x8.clone(), step.clone(), wq, s, z), want)


def test_norm_and_product_in_a_graph_and_on_another_stream():
    t = torch()
    say("norm, q8 and product captured")
    M, N, K = 5, 768, 1024
    c = synth.uniform_case(92, M, N, K, 4)
    wq, s, z = q.pack(dev(c["codes"]), 4), dev(c["scales"]), q.pack_zeros(dev(c["zeros"]), 4)
    x, r, w, y, h = _inputs(M, K, t.float16, 7)
    x8, st = t.empty(M, K, dtype=t.int8, device="cuda"), t.empty(M, device="cuda")
    out = t.empty(M, N, dtype=t.float16, device="cuda")

    def run():
        q.rms_norm_q8(x, w, residual=r, out=x8, scales=st, residual_out=h)
        q.w4a8_rows(x8, st, wq, s, z, out=out)
        q.rms_norm(h, w, out=y)

    run()
    t.cuda.synchronize()
    eager = [out.clone(), y.clone()]
    side = t.cuda.Stream()
    side.wait_stream(t.cuda.current_stream())
    with t.cuda.stream(side):
        run()
    t.cuda.synchronize()
    assert t.equal(out, eager[0]) and t.equal(y, eager[1])
    g = t.cuda.CUDAGraph()
    with t.cuda.graph(g):
        run()
    for _ in range(3):
        for a in (out, y):
            a.fill_(float("nan"))
        t.cuda.synchronize()
        g.replay()
        t.cuda.synchronize()
        assert t.equal(out, eager[0]) and t.equal(y, eager[1])


def test_no_rows():
    t = torch()
    x, w = t.empty(0, 64, device="cuda").half(), t.ones(64, device="cuda").half()
    assert q.rms_norm(x, w).shape == (0, 64)
    assert q.rms_norm(x, w, residual=x)[1].shape == (0, 64)
    assert q.rms_norm_q8(x, w)[1].shape == (0,)
