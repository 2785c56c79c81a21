"""Pools of a cache that lie over one another are refused by the calls that write to them, and only by these."""
import pytest

import gemm_unpack_bit_amd as q
from tests.test_step_abi import FAKE, L, append, cache, calls  # noqa: F401  (L is a fixture)

OVER = [dict(v=FAKE * 10), dict(v=FAKE * 10 + 4096), dict(v_exps=FAKE * 16), dict(k_exps=FAKE * 17 + 32), dict(k_exps=FAKE * 10 + 256),
        dict(v_exps=FAKE * 11), dict(v_exps=FAKE * 10)]


@pytest.mark.parametrize("name", ["append", "fork", "compact"])
@pytest.mark.parametrize("bad", OVER)
def test_8_bits(L, name, bad):  # noqa: F811
    if name == "fork":
        from tests.test_step_abi import b, v

        other = cache(True, tables=FAKE * 30, lens=FAKE * 31, **bad)
        got = L.qgemv_kv8_fork(b(cache(True, **bad)), v(FAKE * 20), b(other), v(FAKE * 22), 1 << 20, v(0))
    else:
        got = calls(L)[name](cache(True, **bad))
    assert got == q.ERR_VALUE


def test_append_to_16_bits(L):  # noqa: F811
    for bad in (dict(v=FAKE * 10), dict(v=FAKE * 10 + 4096)):
        assert append(L, False, c=cache(False, **bad)) == q.ERR_VALUE
    assert append(L, False, c=cache(False, v=FAKE * 10 + 2 * 10 * 16 * 2 * 64 * 2), n=0) == q.OK  # side by side


def test_reads_do_not_mind(L):  # noqa: F811
    from tests.test_step_abi import b, heads, v

    c = cache(True, v=FAKE * 10, v_exps=FAKE * 16)
    assert L.qgemv_kv8_read(0, b(c), 1, 0, v(FAKE * 20), v(FAKE * 21), heads(1), heads(2), v(0)) == q.OK
    assert L.qgemv_attn_tree8(0, b(c), 1, 0, 4, 0.1, heads(1), v(FAKE * 20), v(FAKE * 21), v(0), 0, heads(4), v(FAKE * 60), 1 << 40,
                              v(0)) == q.OK
