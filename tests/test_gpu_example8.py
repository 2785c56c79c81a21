"""The example's serving loop over a cache of 8 bits: it runs, and its rows and pages come out whole."""
import pytest

pytestmark = pytest.mark.gpu

pytest.importorskip("gemm_unpack_bit_amd")


@pytest.mark.parametrize("seed,lengths,ahead", [(1, (37, 5, 120), 4), (3, (1, 16, 64, 3), 7)])
def test_decode_layers_over_a_cache_of_8_bits(seed, lengths, ahead):
    import torch

    from examples import decode_layers as ex
    from tests.gpu_util import say

    say("decode_layers8", seed, lengths, ahead)
    r = ex.main(seed, lengths, ahead, cache_type=torch.float8_e4m3fn)
    assert r["status"] == 0
    # every round accepts at least the roots of the trees
    assert all(n >= 1 for a in r["accepted"] for n in a)
    assert r["lens"] == r["texts"] == [n + 1 + sum(a[b] for a in r["accepted"]) for b, n in enumerate(lengths)]
    # no page is shared or lost at the end
    assert r["pages"] == r["refs"] == sum(-(-n // ex.PAGE) for n in r["lens"])
    assert r["difference"] == r["difference"] and r["difference"] < float("inf")
