"""The ends of the ranges of the attention and cache calls: what lies past them
is refused on the host, before anything is enqueued, so these need no GPU."""
import pytest

import gemm_unpack_bit_amd as q
from tests.test_attn_abi import FAKE, L, cache, calls, heads, prompt, v  # noqa: F401 (L is a fixture)

KEYS_MAX = (1 << 31) - 1024


def test_keys_of_a_row_end_before_32_bits_do(L):  # noqa: F811
    """The kernels look up to a few hundred keys past a row's last one, in 32 bits."""
    one = dict(tokens=0, hk=heads(2, token=0), hv=heads(3, token=0))
    assert prompt(L, tokens_k=KEYS_MAX, **one) == q.OK
    assert prompt(L, tokens_k=KEYS_MAX + 1, **one) == q.ERR_SHAPE
    assert prompt(L, tokens_k=(1 << 31) - 1, **one) == q.ERR_SHAPE
    assert L.qgemv_attn_prompt_workspace_bytes(64, KEYS_MAX + 1, 1, 8, 8, 128) == 0
    for page in (16, 256):
        most = KEYS_MAX // page
        none = cache(page_size=page, max_pages=most, rows=0)  # (no rows: nothing to do)
        far = cache(page_size=page, max_pages=most + 1, rows=0)
        for name in ("reserve", "write", "compact", "tree"):
            assert calls(L)[name](none) == q.OK, name
        for name in ("reserve", "write", "fork", "compact", "tree"):
            assert calls(L)[name](far) == q.ERR_SHAPE, name


def far(n):
    return n << 41  # (spans of up to 2 TB do not meet)


def test_work_that_64_bits_do_not_count(L):  # noqa: F811
    """The work of all rows is added up on the device.  Offsets that go up and down give every row all tokens: the sums
    have to hold that, and sizes for which they would not are refused."""
    import ctypes

    b = ctypes.byref
    c = cache(heads_kv=512, layers=1, rows=65535, page_size=256, max_pages=KEYS_MAX // 256, k=far(1), v=far(2),
              tables=far(3), lens=far(4), refs=far(5), status=far(6))
    tree = lambda n: L.qgemv_attn_tree(0, b(c), 0, n, 512, 0.1, b(heads(0, 512 * 64, 64, far(7))), v(far(8)), v(far(9)), v(0), 0,  # noqa: E731
                                       b(heads(0, 512 * 64, 64, far(10))), v(far(11)), 0, v(0))
    assert tree(1 << 21) == q.ERR_SHAPE
    assert tree(1 << 9) == q.ERR_WORKSPACE  # (every check before the workspace's is passed)
    # a million rows of few queries each
    prompt_ = lambda keys: prompt(L, tokens=1 << 23, tokens_k=keys, batch=1 << 20, nh=32, kv=32, wsb=0, cu=far(8),  # noqa: E731
                                  cuk=far(9), ws=far(11), hq=heads(0, 32 * 64, 64, far(7)), ho=heads(0, 32 * 64, 64, far(10)),
                                  hk=heads(0, 0, 64, far(1)), hv=heads(0, 0, 64, far(2)))
    assert prompt_(KEYS_MAX) == q.ERR_SHAPE
    assert prompt_(1 << 20) == q.ERR_WORKSPACE


def test_no_call_depends_on_a_source_of_randomness_that_throws(L):  # noqa: F811
    """std::random_device throws where the system has no random numbers to give; nothing may leave a C entry that way."""
    import shutil
    import subprocess

    nm = shutil.which("nm")
    if nm is None:
        pytest.skip("needs nm")
    names = subprocess.run([nm, "-D", "--undefined-only", q.LIB_PATH], stdout=subprocess.PIPE, check=True, text=True).stdout
    assert "random_device" not in names


def test_what_a_cache_call_writes_is_apart_from_the_rest(L):  # noqa: F811
    """Positions, the workspace and the cache's state: none inside another, and none inside what the call reads."""
    import ctypes

    b, VALUE = ctypes.byref, q.ERR_VALUE
    at = {n: getattr(cache(), n) for n in ("k", "v", "tables", "lens", "refs", "status")}
    state = [dict(tables=at["lens"]), dict(tables=at["refs"]), dict(lens=at["refs"] + 16), dict(status=at["lens"] + 8),
             dict(refs=at["k"] + 64), dict(tables=at["v"] + 128)]
    reserve = lambda c=None, cu=FAKE * 20, pos=FAKE * 21, ws=FAKE * 22: L.qgemv_kv_reserve(  # noqa: E731
        b(c or cache()), v(cu), v(pos), v(ws), 1 << 20, v(0))
    for s in state:
        assert reserve(cache(**s)) == VALUE, s
    for x in at.values():
        assert reserve(pos=x) == VALUE and reserve(ws=x) == VALUE
    for n in ("tables", "lens", "refs", "status"):
        assert reserve(cu=at[n]) == VALUE
    assert reserve(pos=FAKE * 20 + 12) == VALUE and reserve(ws=FAKE * 20) == VALUE and reserve(ws=FAKE * 21) == VALUE
    other = dict(tables=FAKE * 30, lens=FAKE * 31)
    fork = lambda c=None, o=None, p=FAKE * 20, ws=FAKE * 22: L.qgemv_kv_fork(  # noqa: E731
        b(c or cache()), v(p), b(o or cache(**other)), v(ws), 1 << 20, v(0))
    for s in state[2:4]:
        assert fork(cache(**s), cache(**{**other, **s})) == VALUE, s
    for x in list(at.values()) + [FAKE * 30, FAKE * 31]:
        assert fork(ws=x) == VALUE
        if x not in (at["tables"], at["lens"]):  # (these are only read)
            assert fork(p=x) == VALUE
    assert fork(ws=FAKE * 20) == VALUE
    assert fork(o=cache(tables=FAKE * 30, lens=at["refs"])) == VALUE
    assert fork(o=cache(tables=at["k"], lens=FAKE * 31)) == VALUE
    assert fork(o=cache(tables=FAKE * 30, lens=FAKE * 30 + 16)) == VALUE
    compact = lambda c=None, pos=FAKE * 20, keep=FAKE * 21, count=FAKE * 23, ws=FAKE * 22: L.qgemv_kv_compact(  # noqa: E731
        b(c or cache()), v(pos), v(keep), 4, v(count), v(ws), 1 << 20, v(0))
    for s in state:
        assert compact(cache(**s)) == VALUE, s
    for n, x in at.items():
        assert compact(ws=x) == VALUE
        if n != "lens":  # (a row's length is written when its position and count are read)
            assert compact(pos=x) == VALUE and compact(count=x) == VALUE and compact(keep=x) == VALUE
    for x in (FAKE * 20, FAKE * 21, FAKE * 23):
        assert compact(ws=x) == VALUE
    write = lambda c=None, cu=FAKE * 20, pos=FAKE * 21: L.qgemv_kv_write(  # noqa: E731
        b(c or cache()), 1, 5, b(heads(1, 128)), b(heads(2, 128)), v(cu), v(pos), v(0))
    for x in (at["k"], at["v"]):
        assert write(cu=x) == VALUE and write(pos=x) == VALUE and write(cache(tables=x)) == VALUE
    tree = lambda o=4, ws=FAKE * 60: L.qgemv_attn_tree(  # noqa: E731
        0, b(cache()), 1, 5, 4, 0.1, b(heads(1)), v(FAKE * 20), v(FAKE * 21), v(0), 0, b(heads(o)), v(ws), 1 << 40, v(0))
    for n in ("lens", "refs", "status"):
        assert tree(o=at[n] // FAKE) == VALUE and tree(ws=at[n]) == VALUE


def test_what_is_empty_overlaps_nothing(L):  # noqa: F811
    assert prompt(L, tokens=0, ho=heads(0, data=FAKE * 2 + 128)) == q.OK  # no output, "inside" the keys


def test_a_write_of_more_tokens_than_a_launch_has_waves(L):  # noqa: F811
    import ctypes

    b, c = ctypes.byref, cache(rows=1)
    write = lambda n: L.qgemv_kv_write(b(c), 1, n, b(heads(1, 0)), b(heads(2, 0)), v(FAKE * 20), v(FAKE * 21), v(0))  # noqa: E731
    most = (1 << 26) - 4  # (a wave a token, under 2^32 threads)
    assert write(most + 1) == q.ERR_SHAPE and write((1 << 31) - 1) == q.ERR_SHAPE


def test_strides_of_single_tokens_and_heads_do_not_count(L):  # noqa: F811
    """One token of a padded row, one head of a wider array: the stride of a dimension of one leads nowhere."""
    import ctypes

    b = ctypes.byref
    h = lambda at, token, head: heads(at, token, head)  # noqa: E731
    for token in (260, -8, 1 << 60, 1 << 27):
        one = dict(tokens=1, tokens_k=1, batch=1, wsb=0, hq=h(1, token, 64), hk=h(2, token, 64), hv=h(3, token, 64), ho=h(4, token, 64))
        assert prompt(L, **one) == q.ERR_WORKSPACE, token  # (every check before the workspace's is passed)
        one = dict(tokens=9, tokens_k=9, nh=1, kv=1, batch=1, wsb=0, hq=h(1, 64, token), hk=h(2, 64, token), hv=h(3, 64, token),
                   ho=h(4, 64, token))
        assert prompt(L, **one) == q.ERR_WORKSPACE, token
        c = cache(rows=0)
        assert L.qgemv_attn_tree(0, b(c), 0, 1, 4, 0.1, b(h(1, token, 64)), v(FAKE * 20), v(FAKE * 21), v(0), 0, b(h(4, token, 64)),
                                 v(0), 0, v(0)) == q.OK
        assert L.qgemv_kv_write(b(c), 0, 1, b(h(1, token, 64)), b(h(2, token, 64)), v(FAKE * 20), v(FAKE * 21), v(0)) == q.OK
    assert prompt(L, tokens=2, tokens_k=2, hq=h(1, 260, 64)) == q.ERR_ALIGN
    assert prompt(L, tokens=2, tokens_k=2, hk=h(2, 256, -8)) == q.ERR_SHAPE
