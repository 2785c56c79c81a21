"""The example that runs the attention and cache calls with the packed-weight
products, as a serving loop does, ends with a cache that agrees with one prompt."""
import pytest

pytestmark = pytest.mark.gpu

pytest.importorskip("gemm_unpack_bit_amd")


@pytest.mark.parametrize("seed,lengths,ahead", [(1, (37, 5, 120), 4), (2, (1, 16, 64, 3), 7)])
def test_decode_layers(seed, lengths, ahead):
    from examples import decode_layers as ex
    from tests.gpu_util import say

    say("decode_layers", seed, lengths, ahead)
    r = ex.main(seed, lengths, ahead)
    assert r["status"] == 0
    # scouted tokens are what the layers say themselves, so trees are accepted beyond their roots
    assert sum(map(sum, r["accepted"])) > 2 * len(lengths)
    assert r["lens"] == r["texts"] == [n + 1 + sum(a[b] for a in r["accepted"]) for b, n in enumerate(lengths)]
    # no page is shared or lost at the end
    assert r["pages"] == r["refs"] == sum(-(-n // ex.PAGE) for n in r["lens"])
    # Both ways round to fp16 about 8 times a layer and twice outside the layers, each a relative 2^-11 at most; a
    # wrong key or position changes the logits by the order of themselves.
    assert r["difference"] < 2 * (8 * ex.LAYERS + 2) * 2.0 ** -11
