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
