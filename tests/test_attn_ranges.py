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
