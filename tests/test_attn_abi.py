"""Refusals of the attention and cache calls: every check runs on the host
before anything is enqueued, so these need no GPU."""
import ctypes

import pytest

import gemm_unpack_bit_amd as q

FAKE = 0x100000  # 16-byte aligned, never dereferenced: every call below fails validation first
v = ctypes.c_void_p


class Heads(ctypes.Structure):
    _fields_ = [("data", v), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("layers", "pages", "page_size", "heads_kv", "head_dim", "rows", "max_pages")]
    _fields_ += [(n, v) for n in ("k", "v", "tables", "lens", "refs", "status")]


@pytest.fixture(scope="module")
def L():
    import os

    if not os.path.exists(q.LIB_PATH):
        pytest.skip("library not built")
    return q.lib()


def heads(at, token=256, head=64, data=None):
    return Heads(FAKE * at if data is None else data, token, head)


def prompt(L, dtype=0, tokens=100, tokens_k=100, batch=2, nh=4, kv=2, dim=64, scale=0.1, hq=None, hk=None, hv=None,
           ho=None, cu=FAKE * 50, cuk=FAKE * 51, ws=FAKE * 60, wsb=1 << 40):
    b = ctypes.byref
    return L.qgemv_attn_prompt(dtype, 1, tokens, tokens_k, batch, nh, kv, dim, scale, b(hq or heads(1)), b(hk or heads(2)),
                               b(hv or heads(3)), v(cu), v(cuk), b(ho or heads(4)), v(ws), wsb, v(0))


def test_prompt(L):
    assert prompt(L, hq=heads(1, data=0)) == q.ERR_NULL
    assert prompt(L, ho=heads(1, data=0)) == q.ERR_NULL
    assert prompt(L, cu=0) == q.ERR_NULL
    assert prompt(L, dtype=2) == q.ERR_UNSUPPORTED
    assert prompt(L, dim=96) == q.ERR_UNSUPPORTED
    assert prompt(L, dim=32) == q.ERR_UNSUPPORTED
    assert prompt(L, nh=5) == q.ERR_SHAPE
    assert prompt(L, kv=0) == q.ERR_SHAPE
    assert prompt(L, tokens=-1) == q.ERR_SHAPE
    assert prompt(L, tokens_k=-1) == q.ERR_SHAPE
    assert prompt(L, batch=-1) == q.ERR_SHAPE
    assert prompt(L, tokens=1 << 30) == q.ERR_SHAPE
    assert prompt(L, hq=heads(1, token=-256)) == q.ERR_SHAPE
    assert prompt(L, hk=heads(2, token=1 << 60)) == q.ERR_SHAPE
    assert prompt(L, ho=heads(4, token=128)) == q.ERR_SHAPE        # tokens of the output overlap
    assert prompt(L, ho=heads(4, token=256, head=0)) == q.ERR_SHAPE
    assert prompt(L, scale=float("nan")) == q.ERR_VALUE
    assert prompt(L, scale=float("inf")) == q.ERR_VALUE
    assert prompt(L, scale=-1.0) == q.ERR_VALUE
    assert prompt(L, hq=heads(1, data=FAKE + 8)) == q.ERR_ALIGN
    assert prompt(L, hk=heads(2, token=260)) == q.ERR_ALIGN
    assert prompt(L, hv=heads(3, head=68)) == q.ERR_ALIGN
    assert prompt(L, cu=FAKE * 50 + 2) == q.ERR_ALIGN
    assert prompt(L, ho=heads(1)) == q.ERR_VALUE                   # the output over the queries
    assert prompt(L, ho=heads(0, data=FAKE * 2 + 64 * 100)) == q.ERR_VALUE  # ... inside the keys
    assert prompt(L, tokens=4, tokens_k=4, ws=FAKE) == q.ERR_VALUE  # the workspace over the queries
    assert prompt(L, tokens=4, tokens_k=4, ws=0) == q.ERR_WORKSPACE
    assert prompt(L, tokens=4, tokens_k=4, wsb=100) == q.ERR_WORKSPACE
    assert prompt(L, tokens=4, tokens_k=4, ws=FAKE * 60 + 8) == q.ERR_ALIGN
    assert prompt(L, tokens=0) == q.OK and prompt(L, batch=0) == q.OK  # nothing to do


def test_workspaces(L):
    assert L.qgemv_attn_prompt_workspace_bytes(1 << 16, 1 << 16, 1, 64, 8, 128) == 0  # enough tiles: no split
    assert L.qgemv_attn_prompt_workspace_bytes(4, 4, 1, 64, 8, 128) > 0
    for bad in ((-1, 4, 1, 8, 8, 128), (4, -1, 1, 8, 8, 128), (4, 4, 0, 8, 8, 128), (4, 4, 1, 8, 3, 128), (4, 4, 1, 8, 8, 80)):
        assert L.qgemv_attn_prompt_workspace_bytes(*bad) == 0
    assert L.qgemv_attn_tree_workspace_bytes(1, 1, 32, 8, 128) > 0
    assert L.qgemv_attn_tree_workspace_bytes(64, 1, 32, 8, 128) > 0
    assert L.qgemv_attn_tree_workspace_bytes(0, 1, 32, 8, 128) == 0
    assert L.qgemv_kv_workspace_bytes(3, 100) >= 4 * (100 + 2 * 3)
    assert L.qgemv_kv_workspace_bytes(3, 0) == 0 and L.qgemv_kv_workspace_bytes(-1, 4) == 0


def cache(**k):
    d = dict(layers=2, pages=10, page_size=16, heads_kv=2, head_dim=64, rows=3, max_pages=4, k=FAKE * 10, v=FAKE * 11,
             tables=FAKE * 12, lens=FAKE * 13, refs=FAKE * 14, status=FAKE * 15)
    d.update(k)
    return Cache(*[d[n] for n, _ in Cache._fields_])


def calls(L):
    """Every cache call as a function of its cache."""
    b, h = ctypes.byref, heads
    return {
        "reserve": lambda c: L.qgemv_kv_reserve(b(c), v(FAKE * 20), v(FAKE * 21), v(FAKE * 22), 1 << 20, v(0)),
        "write": lambda c: L.qgemv_kv_write(b(c), 1, 5, b(h(1, 128)), b(h(2, 128)), v(FAKE * 20), v(FAKE * 21), v(0)),
        "fork": lambda c: L.qgemv_kv_fork(b(c), v(FAKE * 20), b(cache(tables=FAKE * 30, lens=FAKE * 31)), v(FAKE * 22), 1 << 20, v(0)),
        "compact": lambda c: L.qgemv_kv_compact(b(c), v(FAKE * 20), v(FAKE * 21), 4, v(FAKE * 23), v(FAKE * 22), 1 << 20, v(0)),
        "tree": lambda c: L.qgemv_attn_tree(0, b(c), 1, 5, 4, 0.1, b(h(1)), v(FAKE * 20), v(FAKE * 21), v(0), 0, b(h(4)),
                                            v(FAKE * 60), 1 << 40, v(0)),
    }


BAD = [(dict(k=0), "ERR_NULL"), (dict(tables=0), "ERR_NULL"), (dict(head_dim=80), "ERR_UNSUPPORTED"),
       (dict(page_size=8), "ERR_UNSUPPORTED"), (dict(page_size=48), "ERR_UNSUPPORTED"), (dict(page_size=512), "ERR_UNSUPPORTED"),
       (dict(pages=0), "ERR_SHAPE"), (dict(layers=0), "ERR_SHAPE"), (dict(max_pages=0), "ERR_SHAPE"),
       (dict(rows=-1), "ERR_SHAPE"), (dict(rows=65536), "ERR_SHAPE"), (dict(heads_kv=0), "ERR_SHAPE"),
       (dict(max_pages=1 << 27), "ERR_SHAPE"), (dict(k=FAKE * 10 + 8), "ERR_ALIGN"), (dict(tables=FAKE * 12 + 2), "ERR_ALIGN")]


@pytest.mark.parametrize("name", ["reserve", "write", "fork", "compact", "tree"])
@pytest.mark.parametrize("bad,want", BAD)
def test_every_call_checks_its_cache(L, name, bad, want):
    assert calls(L)[name](cache(**bad)) == getattr(q, want)


@pytest.mark.parametrize("name", ["reserve", "fork", "compact"])
@pytest.mark.parametrize("bad,want", [(dict(refs=0), "ERR_NULL"), (dict(lens=0), "ERR_NULL"), (dict(status=0), "ERR_NULL"),
                                      (dict(refs=FAKE * 14 + 1), "ERR_ALIGN")])
def test_state_is_checked(L, name, bad, want):
    assert calls(L)[name](cache(**bad)) == getattr(q, want)


def test_other_arguments(L):
    b, h = ctypes.byref, heads
    c = cache()
    r = lambda cu=FAKE * 20, pos=FAKE * 21, ws=FAKE * 22, n=1 << 20: L.qgemv_kv_reserve(b(c), v(cu), v(pos), v(ws), n, v(0))
    assert r(cu=0) == q.ERR_NULL and r(pos=0) == q.ERR_NULL
    assert r(cu=FAKE + 1) == q.ERR_ALIGN and r(ws=FAKE * 22 + 4) == q.ERR_ALIGN
    assert r(ws=0) == q.ERR_WORKSPACE and r(n=16) == q.ERR_WORKSPACE
    w = lambda layer=0, n=5, hk=None, hv=None: L.qgemv_kv_write(b(c), layer, n, b(hk or h(1, 128)), b(hv or h(2, 128)),
                                                              v(FAKE * 20), v(FAKE * 21), v(0))
    assert w(layer=2) == q.ERR_SHAPE and w(layer=-1) == q.ERR_SHAPE and w(n=-1) == q.ERR_SHAPE
    assert w(hk=h(1, data=0)) == q.ERR_NULL and w(hk=h(1, 130)) == q.ERR_ALIGN
    assert w(hv=h(10)) == q.ERR_VALUE  # new values inside the pool
    assert w(n=0) == q.OK
    f = lambda o, p=FAKE * 20: L.qgemv_kv_fork(b(c), v(p), b(o), v(FAKE * 22), 1 << 20, v(0))
    other = dict(tables=FAKE * 30, lens=FAKE * 31)
    assert f(cache(**other), p=0) == q.ERR_NULL
    assert f(cache(**other, pages=9)) == q.ERR_SHAPE and f(cache(**other, max_pages=5)) == q.ERR_SHAPE
    assert f(cache()) == q.ERR_VALUE                       # its own tables
    assert f(cache(**other, refs=FAKE * 32)) == q.ERR_VALUE  # another pool's state
    k = lambda keep=FAKE * 21, n=4: L.qgemv_kv_compact(b(c), v(FAKE * 20), v(keep), n, v(FAKE * 23), v(FAKE * 22), 1 << 20, v(0))
    assert k(keep=0) == q.ERR_NULL and k(n=-1) == q.ERR_SHAPE
    t = lambda dtype=0, layer=1, n=5, nh=4, s=0.1, mask=0, words=0, ho=None, ws=FAKE * 60, wsb=1 << 40: L.qgemv_attn_tree(
        dtype, b(c), layer, n, nh, s, b(h(1)), v(FAKE * 20), v(FAKE * 21), v(mask), words, b(ho or h(4)), v(ws), wsb, v(0))
    assert t(dtype=7) == q.ERR_UNSUPPORTED and t(layer=2) == q.ERR_SHAPE and t(nh=3) == q.ERR_SHAPE
    assert t(mask=FAKE * 40) == q.ERR_SHAPE and t(words=1) == q.ERR_SHAPE
    assert t(mask=FAKE * 40 + 4, words=1) == q.ERR_ALIGN
    assert t(s=float("nan")) == q.ERR_VALUE and t(ho=h(12)) == q.ERR_VALUE and t(ho=h(10)) == q.ERR_VALUE
    assert t(ws=0) == q.ERR_WORKSPACE and t(wsb=64) == q.ERR_WORKSPACE
    assert t(n=0) == q.OK


def test_python_arguments():
    torch = pytest.importorskip("torch")
    x = torch.zeros(4, 2, 64, dtype=torch.float16)
    with pytest.raises(TypeError):
        q.attn_prompt(x, x, x, torch.zeros(2, dtype=torch.int32))  # not on the GPU
    with pytest.raises(TypeError):
        q.KvCache(x, x, x, x, x)
    with pytest.raises(AttributeError):
        q.no_such_name
