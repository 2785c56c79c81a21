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
