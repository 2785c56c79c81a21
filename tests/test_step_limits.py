"""Which sizes the sampling and append calls take, and which they refuse, on both sides of the limits that their headers
name.  Calls that pass the check of sizes stop at a later one (no workspace, a bad address), so nothing is enqueued."""
import ctypes
import itertools
import os

import pytest

import gemm_unpack_bit_amd as q

FAKE = 0x100000  # 16-byte aligned, never dereferenced
v = ctypes.c_void_p


@pytest.fixture(scope="module")
def L():
    if not os.path.exists(q.LIB_PATH):
        pytest.skip("library not built")
    return q.lib()


def sample(L, n, vocab, row):
    return L.qgemv_sample(2, n, vocab, v(1 << 62), row, v(FAKE), v(0), v(0), v(0), v(0), v(FAKE * 200), v(0), 0, v(0))


def test_sample(L):
    edges = []
    for vocab in (1, 2047, 2048, 16384, 16385, 32768, 32769, 151643, 1 << 20, (1 << 21) - 1, 1 << 21):
        most = min((1 << 21) - 1, ((1 << 23) - 1) // -(-vocab // 16384))
        edges += [(1, vocab), (7, vocab), (1000, vocab), (most - 1, vocab), (most, vocab), (most + 1, vocab), (1 << 21, vocab)]
    edges += list(itertools.product((1, 30, 1023, 8191, 8192, 100000, 1200000), (100, 8000, 20001, 300001)))
    for rows, vocab in edges:
        fits = rows < 1 << 21 and rows * -(-vocab // 16384) < 1 << 23
        assert (L.qgemv_sample_workspace_bytes(rows, vocab) > 0) == fits, (rows, vocab)
        assert sample(L, rows, vocab, vocab) == (q.ERR_WORKSPACE if fits else q.ERR_SHAPE), (rows, vocab)


def test_sample_strides(L):
    assert sample(L, 2, 1000, 1 << 40) == q.ERR_WORKSPACE and sample(L, 2, 1000, (1 << 40) + 1) == q.ERR_SHAPE
    assert sample(L, 180000, 1000, 1 << 40) == q.ERR_WORKSPACE and sample(L, 182000, 1000, 1 << 40) == q.ERR_SHAPE
    assert sample(L, 2, 1000, 0) == q.ERR_WORKSPACE and sample(L, 2, 1000, -1) == q.ERR_SHAPE
    assert sample(L, 1, 1000, -1) == q.ERR_WORKSPACE  # (that of a single row is not looked at)


class Heads(ctypes.Structure):
    _fields_ = [("data", v), ("token", ctypes.c_int64), ("head", ctypes.c_int64)]


class Cache(ctypes.Structure):
    _fields_ = [(n, ctypes.c_int) for n in ("layers", "pages", "page_size", "heads_kv", "head_dim", "rows", "max_pages")]
    _fields_ += [(n, v) for n in ("k", "v", "tables", "lens", "refs", "status")]


class Cache8(ctypes.Structure):
    _fields_ = Cache._fields_[:9] + [("k_exps", v), ("v_exps", v)] + Cache._fields_[9:]


def cache(eight, rows, kv):
    kind = Cache8 if eight else Cache
    return ctypes.byref(kind(1, 10, 16, kv, 64, rows, 4, *[FAKE * (10 + i) for i in range(8 if eight else 6)]))


@pytest.mark.parametrize("eight", [False, True])
def test_append(L, eight):
    call = L.qgemv_kv8_append if eight else L.qgemv_kv_append
    for heads, kv, rows in ((0, 1, 1), (8, 1, 300), (32, 8, 48), (64, 8, 65535), (1000, 100, 5000)):
        most = ((1 << 29) - 65 - 32 * rows * kv) // (heads + 2 * kv + 8)
        h = lambda n, at: ctypes.byref(Heads(FAKE + at, n * 64, 64))  # noqa: E731
        for tokens in (most - 1, most, most + 1, most + 2):
            got = call(0, cache(eight, rows, kv), 0, tokens, heads, h(heads, 0), h(kv, 8), h(kv, 0), v(FAKE), v(FAKE), v(0), 0, 0, v(0),
                       h(heads, 0), v(0))
            assert got == (q.ERR_ALIGN if tokens <= most else q.ERR_SHAPE), (heads, kv, rows, tokens)


@pytest.mark.parametrize("eight", [False, True])
def test_read(L, eight):
    h = lambda at: ctypes.byref(Heads(FAKE + at, 128, 64))  # noqa: E731
    for tokens, want in (((1 << 26) - 4, q.ERR_ALIGN), ((1 << 26) - 3, q.ERR_SHAPE)):
        more = (cache(eight, 3, 2), 0, tokens, v(FAKE), v(FAKE), h(8), h(0), v(0))
        assert (L.qgemv_kv8_read(0, *more) if eight else L.qgemv_kv_read(*more)) == want
