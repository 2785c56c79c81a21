"""Refusals of the norm, sampling, append and 8-bit cache calls: every check
runs on the host before anything is enqueued, so these need no GPU."""
import ctypes
import os

import pytest

import gemm_unpack_bit_amd as q

FAKE = 0x100000  # 16-byte aligned, never dereferenced: every call below fails validation first
v = ctypes.c_void_p
b = ctypes.byref


class Rows(ctypes.Structure):
    _fields_ = [("data", v), ("row", ctypes.c_int64)]


class Heads(ctypes.Structure):
    _fields_ = [("data", v), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("layers", "pages", "page_size", "heads_kv", "head_dim", "rows", "max_pages")]
    _fields_ += [(n, v) for n in ("k", "v", "tables", "lens", "refs", "status")]


class Cache8(ctypes.Structure):
    _fields_ = Cache._fields_[:9] + [("k_exps", v), ("v_exps", v)] + Cache._fields_[9:]


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(q.LIB_PATH):
        pytest.skip("library not built")
    return q.lib()


def rows(at, row=256, data=None):
    return b(Rows(FAKE * at if data is None else data, row))


def norm(L, q8=False, dtype=0, n=10, dim=256, eps=1e-6, x=None, r=None, w=FAKE * 3, s=None, y=None, y8=FAKE * 6, step=FAKE * 7):
    x = rows(1) if x is None else x
    if q8:
        return L.qgemv_rms_norm_q8(dtype, n, dim, eps, x, r, v(w), s, v(y8), v(step), v(0))
    return L.qgemv_rms_norm(dtype, n, dim, eps, x, r, v(w), s, rows(5) if y is None else y, v(0))


@pytest.mark.parametrize("q8", [False, True])
def test_norm(L, q8):
    f = lambda **k: norm(L, q8, **k)  # noqa: E731
    assert f(x=rows(1, data=0)) == q.ERR_NULL and f(w=0) == q.ERR_NULL
    assert f(r=rows(2)) == q.ERR_NULL and f(s=rows(4)) == q.ERR_NULL          # a residual without its sum, and a sum alone
    assert f(r=rows(2, data=0), s=rows(4)) == q.ERR_NULL
    assert f(dtype=2) == q.ERR_UNSUPPORTED
    assert f(n=-1) == q.ERR_SHAPE and f(dim=0) == q.ERR_SHAPE and f(dim=(1 << 24) + 1) == q.ERR_SHAPE
    assert f(x=rows(1, -1)) == q.ERR_SHAPE and f(x=rows(1, 1 << 41)) == q.ERR_SHAPE
    assert f(r=rows(2), s=rows(4, 255)) == q.ERR_SHAPE                        # rows of the sum overlap
    for eps in (float("nan"), float("inf"), -1e-6):
        assert f(eps=eps) == q.ERR_VALUE
    assert f(x=rows(1, data=FAKE + 1)) == q.ERR_ALIGN and f(w=FAKE * 3 + 1) == q.ERR_ALIGN
    assert f(r=rows(2), s=rows(3)) == q.ERR_VALUE                             # the sum over the weights
    assert f(r=rows(2), s=rows(0, data=FAKE + 2)) == q.ERR_VALUE              # ... beside itself over x
    assert f(r=rows(2), s=rows(1, 257)) == q.ERR_VALUE                        # ... over x by another stride
    assert f(n=0) == q.OK
    if q8:
        assert f(y8=0) == q.ERR_NULL and f(step=0) == q.ERR_NULL and f(step=FAKE * 7 + 2) == q.ERR_ALIGN
        assert f(y8=FAKE) == q.ERR_VALUE and f(step=FAKE * 6) == q.ERR_VALUE and f(step=FAKE) == q.ERR_VALUE
        assert f(r=rows(2), s=rows(6)) == q.ERR_VALUE
    else:
        assert f(y=rows(5, data=0)) == q.ERR_NULL and f(y=rows(5, 200)) == q.ERR_SHAPE
        assert f(y=rows(3)) == q.ERR_VALUE and f(y=rows(0, data=FAKE + 512)) == q.ERR_VALUE
        assert f(r=rows(2), s=rows(5)) == q.ERR_VALUE                         # both results in one place
        assert L.qgemv_rms_norm(0, 1, 8, 0.0, rows(1), None, v(FAKE), None, None, v(0)) == q.ERR_NULL


def test_ready_rows(L):
    f = lambda M=4, N=64, K=256, x=FAKE, s=FAKE * 2, w=FAKE * 3, sc=FAKE * 4, z=FAKE * 5, y=FAKE * 6: L.qgemv_w4a8_rows(  # noqa: E731
        M, N, K, v(x), v(s), v(w), v(sc), v(z), v(y), v(0))
    for name in ("x", "s", "w", "sc", "z", "y"):
        assert f(**{name: 0}) == q.ERR_NULL
    assert f(M=0) == q.ERR_SHAPE and f(M=17) == q.ERR_SHAPE and f(K=100) == q.ERR_SHAPE and f(N=0) == q.ERR_SHAPE
    assert f(x=FAKE + 8) == q.ERR_ALIGN and f(s=FAKE * 2 + 2) == q.ERR_ALIGN and f(y=FAKE * 6 + 1) == q.ERR_ALIGN
    for at in (1, 2, 3, 4, 5):
        assert f(y=FAKE * at) == q.ERR_VALUE


def test_sample(L):
    f = lambda t=2, n=4, vocab=1000, x=FAKE, row=1000, u=FAKE * 2, temp=0, k=0, p=0, low=0, out=FAKE * 7, ws=FAKE * 8, wsb=1 << 30: (  # noqa: E731
        L.qgemv_sample(t, n, vocab, v(x), row, v(u), v(temp), v(k), v(p), v(low), v(out), v(ws), wsb, v(0)))
    assert f(x=0) == q.ERR_NULL and f(u=0) == q.ERR_NULL and f(out=0) == q.ERR_NULL
    assert f(t=3) == q.ERR_UNSUPPORTED and f(t=-1) == q.ERR_UNSUPPORTED
    assert f(n=-1) == q.ERR_SHAPE and f(vocab=0) == q.ERR_SHAPE and f(vocab=(1 << 21) + 1) == q.ERR_SHAPE
    assert f(n=1 << 21) == q.ERR_SHAPE and f(row=-1) == q.ERR_SHAPE and f(row=1 << 41) == q.ERR_SHAPE
    assert f(x=FAKE + 2) == q.ERR_ALIGN and f(t=0, x=FAKE + 1) == q.ERR_ALIGN and f(u=FAKE * 2 + 1) == q.ERR_ALIGN
    assert f(k=FAKE * 3 + 2) == q.ERR_ALIGN and f(out=FAKE * 7 + 2) == q.ERR_ALIGN and f(ws=FAKE * 8 + 4) == q.ERR_ALIGN
    assert f(out=FAKE) == q.ERR_VALUE and f(out=FAKE * 2) == q.ERR_VALUE and f(k=FAKE * 7) == q.ERR_VALUE
    assert f(ws=FAKE) == q.ERR_VALUE and f(p=FAKE * 8) == q.ERR_VALUE and f(out=FAKE * 8 + 64) == q.ERR_VALUE
    need = L.qgemv_sample_workspace_bytes(4, 1000)
    assert need > 0 and f(ws=0) == q.ERR_WORKSPACE and f(wsb=need - 1) == q.ERR_WORKSPACE
    assert f(n=0) == q.OK
    for bad in ((0, 100), (-1, 100), (4, 0), (4, (1 << 21) + 1), (1 << 22, 1)):
        assert L.qgemv_sample_workspace_bytes(*bad) == 0


def cache(eight, **k):
    d = dict(layers=2, pages=10, page_size=16, heads_kv=2, head_dim=64, rows=3, max_pages=4, k=FAKE * 10, v=FAKE * 11,
             k_exps=FAKE * 16, v_exps=FAKE * 17, tables=FAKE * 12, lens=FAKE * 13, refs=FAKE * 14, status=FAKE * 15)
    d.update(k)
    kind = Cache8 if eight else Cache
    return kind(*[d[n] for n, _ in kind._fields_])


def heads(at, token=512, head=64, data=None):
    return b(Heads(FAKE * at if data is None else data, token, head))


def append(L, eight, c=None, dtype=0, layer=1, n=5, nh=4, hq=None, hk=None, hv=None, cu=FAKE * 20, pos=FAKE * 21, f=FAKE * 22, rot=64,
           at=0, ho=None):
    fn = L.qgemv_kv8_append if eight else L.qgemv_kv_append
    return fn(dtype, b(cache(eight) if c is None else c), layer, n, nh, hq or heads(1), hk or heads(2), hv or heads(3), v(cu), v(pos),
              v(f), rot, 0, v(at), ho or heads(4), v(0))


@pytest.mark.parametrize("eight", [False, True])
def test_append(L, eight):
    f = lambda **k: append(L, eight, **k)  # noqa: E731
    for bad in (dict(hk=heads(0, data=0)), dict(hv=heads(0, data=0)), dict(hq=heads(0, data=0)), dict(ho=heads(0, data=0)), dict(cu=0),
                dict(pos=0), dict(f=0), dict(c=cache(eight, k=0)), dict(c=cache(eight, tables=0))):
        assert f(**bad) == q.ERR_NULL, bad
    assert f(dtype=2) == q.ERR_UNSUPPORTED and f(rot=8) == q.ERR_UNSUPPORTED and f(rot=80) == q.ERR_UNSUPPORTED
    assert f(rot=-16) == q.ERR_UNSUPPORTED and f(c=cache(eight, head_dim=80)) == q.ERR_UNSUPPORTED
    assert f(c=cache(eight, page_size=8)) == q.ERR_UNSUPPORTED
    assert f(layer=2) == q.ERR_SHAPE and f(layer=-1) == q.ERR_SHAPE and f(n=-1) == q.ERR_SHAPE and f(nh=-1) == q.ERR_SHAPE
    assert f(n=1 << 28) == q.ERR_SHAPE and f(c=cache(eight, rows=70000)) == q.ERR_SHAPE
    assert f(ho=heads(4, 128)) == q.ERR_SHAPE and f(hk=heads(2, -8)) == q.ERR_SHAPE
    assert f(hq=heads(1, 260)) == q.ERR_ALIGN and f(hv=heads(0, data=FAKE + 8)) == q.ERR_ALIGN and f(f=FAKE * 22 + 4) == q.ERR_ALIGN
    assert f(at=FAKE * 23 + 2) == q.ERR_ALIGN and f(cu=FAKE * 20 + 2) == q.ERR_ALIGN
    assert f(ho=heads(2)) == q.ERR_VALUE and f(ho=heads(0, data=FAKE * 1 + 128)) == q.ERR_VALUE   # over keys, beside itself over q
    assert f(ho=heads(10)) == q.ERR_VALUE and f(hk=heads(11)) == q.ERR_VALUE and f(ho=heads(12)) == q.ERR_VALUE
    assert f(ho=heads(20)) == q.ERR_VALUE and f(cu=FAKE * 10) == q.ERR_VALUE and f(at=FAKE * 4) == q.ERR_VALUE
    # queries, keys and values of one product: in place is fine, over a neighbour is not
    part = lambda h: heads(0, 512, 64, FAKE + 128 * h)  # noqa: E731
    assert f(hq=part(0), hk=part(4), hv=part(6), ho=part(1)) == q.ERR_VALUE
    assert f(hq=part(0), hk=part(4), hv=part(6), ho=part(4)) == q.ERR_VALUE
    assert f(n=0, hq=part(0), hk=part(4), hv=part(6), ho=part(0)) == q.OK
    assert f(n=0) == q.OK and f(c=cache(eight, rows=0)) == q.OK
    if eight:
        assert f(c=cache(True, k_exps=0)) == q.ERR_NULL and f(c=cache(True, v_exps=0)) == q.ERR_NULL
        assert f(ho=heads(16)) == q.ERR_VALUE and f(hv=heads(17)) == q.ERR_VALUE


@pytest.mark.parametrize("eight", [False, True])
def test_read(L, eight):
    def f(c=None, dtype=0, layer=0, n=5, cu=FAKE * 20, start=FAKE * 21, hk=None, hv=None):
        c, more = b(cache(eight) if c is None else c), (v(cu), v(start), hk or heads(1), hv or heads(2), v(0))
        return L.qgemv_kv8_read(dtype, c, layer, n, *more) if eight else L.qgemv_kv_read(c, layer, n, *more)

    assert f(cu=0) == q.ERR_NULL and f(start=0) == q.ERR_NULL and f(hk=heads(0, data=0)) == q.ERR_NULL
    assert f(c=cache(eight, v=0)) == q.ERR_NULL
    assert f(layer=2) == q.ERR_SHAPE and f(n=-1) == q.ERR_SHAPE and f(n=1 << 27) == q.ERR_SHAPE
    assert f(hk=heads(1, 64)) == q.ERR_SHAPE and f(hv=heads(2, 512, 0)) == q.ERR_SHAPE
    assert f(hk=heads(1, 516)) == q.ERR_ALIGN and f(start=FAKE * 21 + 2) == q.ERR_ALIGN
    assert f(hk=heads(2)) == q.ERR_VALUE and f(hk=heads(10)) == q.ERR_VALUE and f(hv=heads(12)) == q.ERR_VALUE
    assert f(hv=heads(20)) == q.ERR_VALUE and f(n=0) == q.OK
    if eight:
        assert f(dtype=2) == q.ERR_UNSUPPORTED and f(hk=heads(16)) == q.ERR_VALUE


def calls(L):
    return {
        "reserve": lambda c: L.qgemv_kv8_reserve(b(c), v(FAKE * 20), v(FAKE * 21), v(FAKE * 22), 1 << 20, v(0)),
        "append": lambda c: append(L, True, c=c),
        "read": lambda c: L.qgemv_kv8_read(0, b(c), 1, 5, v(FAKE * 20), v(FAKE * 21), heads(1), heads(2), v(0)),
        "fork": lambda c: L.qgemv_kv8_fork(b(c), v(FAKE * 20), b(cache(True, tables=FAKE * 30, lens=FAKE * 31)), v(FAKE * 22), 1 << 20, v(0)),
        "compact": lambda c: L.qgemv_kv8_compact(b(c), v(FAKE * 20), v(FAKE * 21), 4, v(FAKE * 23), v(FAKE * 22), 1 << 20, v(0)),
        "tree": lambda c: L.qgemv_attn_tree8(0, b(c), 1, 5, 4, 0.1, heads(1), v(FAKE * 20), v(FAKE * 21), v(0), 0, heads(4), v(FAKE * 60),
                                             1 << 40, v(0)),
    }


BAD = [(dict(k=0), "ERR_NULL"), (dict(k_exps=0), "ERR_NULL"), (dict(v_exps=0), "ERR_NULL"), (dict(tables=0), "ERR_NULL"),
       (dict(head_dim=96), "ERR_UNSUPPORTED"), (dict(page_size=24), "ERR_UNSUPPORTED"), (dict(page_size=512), "ERR_UNSUPPORTED"),
       (dict(pages=0), "ERR_SHAPE"), (dict(layers=0), "ERR_SHAPE"), (dict(heads_kv=0), "ERR_SHAPE"), (dict(rows=65536), "ERR_SHAPE"),
       (dict(max_pages=1 << 27), "ERR_SHAPE"), (dict(v=FAKE * 11 + 8), "ERR_ALIGN"), (dict(tables=FAKE * 12 + 2), "ERR_ALIGN")]


@pytest.mark.parametrize("name", ["reserve", "append", "read", "fork", "compact", "tree"])
@pytest.mark.parametrize("bad,want", BAD)
def test_every_call_checks_a_cache_of_8_bits(L, name, bad, want):
    assert calls(L)[name](cache(True, **bad)) == getattr(q, want)


@pytest.mark.parametrize("name", ["reserve", "fork", "compact"])
def test_exponents_lie_apart_from_the_state(L, name):
    for bad in (dict(k_exps=FAKE * 12), dict(v_exps=FAKE * 14), dict(k_exps=FAKE * 22)):
        want = q.ERR_VALUE
        assert calls(L)[name](cache(True, **bad)) == want, bad


def test_fork_wants_the_same_exponents(L):
    other = cache(True, tables=FAKE * 30, lens=FAKE * 31, k_exps=FAKE * 40)
    assert L.qgemv_kv8_fork(b(cache(True)), v(FAKE * 20), b(other), v(FAKE * 22), 1 << 20, v(0)) == q.ERR_VALUE


def test_attention_over_8_bits(L):
    c = cache(True)
    t = lambda dtype=0, layer=1, n=5, nh=4, s=0.1, mask=0, words=0, ho=None, ws=FAKE * 60, wsb=1 << 40: L.qgemv_attn_tree8(  # noqa: E731
        dtype, b(c), layer, n, nh, s, heads(1), v(FAKE * 20), v(FAKE * 21), v(mask), words, ho or heads(4), v(ws), wsb, v(0))
    assert t(dtype=2) == q.ERR_UNSUPPORTED and t(layer=2) == q.ERR_SHAPE and t(nh=3) == q.ERR_SHAPE and t(words=1) == q.ERR_SHAPE
    assert t(s=float("nan")) == q.ERR_VALUE and t(ho=heads(10)) == q.ERR_VALUE and t(ho=heads(16)) == q.ERR_VALUE
    assert t(ho=heads(17)) == q.ERR_VALUE and t(ws=FAKE * 16) == q.ERR_VALUE
    assert t(ws=0) == q.ERR_WORKSPACE and t(wsb=64) == q.ERR_WORKSPACE and t(n=0) == q.OK


def test_python_arguments():
    torch = pytest.importorskip("torch")
    x, w, u = torch.zeros(4, 64, dtype=torch.float16), torch.ones(64, dtype=torch.float16), torch.zeros(4)
    for f in (lambda: q.rms_norm(x, w), lambda: q.rms_norm_q8(x, w), lambda: q.sample(x, u), lambda: q.rms_norm(x.float(), w),
              lambda: q.sample(x.int(), u), lambda: q.w4a8_rows(x.to(torch.int8), u, x, x, x)):
        with pytest.raises(TypeError):
            f()
    with pytest.raises(ValueError):
        q.rms_norm(x[0], w)
    pool = torch.zeros(1, 2, 16, 1, 64, dtype=torch.uint8).view(torch.float8_e4m3fn)
    with pytest.raises(TypeError):
        q.KvCache(pool, pool, x, x, x)
