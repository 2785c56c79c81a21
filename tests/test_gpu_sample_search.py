"""GPU tests of the rows that sampling searches from the logits alone: many of them at once, several times over, so that
a row whose waves did not agree on how many elements its search had left would show."""
import numpy as np
import pytest

from tests.gpu_util import say, torch
from tests.test_gpu_sample import check, logits

pytestmark = pytest.mark.gpu

q = pytest.importorskip("gemm_unpack_bit_amd")


@pytest.mark.parametrize("dtype", ["float16", "float32"])
@pytest.mark.parametrize("vocab", [5000, 40007])
def test_searched_rows(vocab, dtype):
    """By count, by weight and by both, where thousands of elements share the bin in which the prefix ends, and where the
    count alone is past the list: 384 rows, their tokens those of the definition, and the same ones in every call."""
    t = torch()
    rows = 384
    x = logits(rows, vocab, dtype, vocab, 0.02)
    x[:, 7] = -60.0                    # the others lie in a few bins of a thousand
    x[1::3] = logits(rows // 3, vocab, dtype, 1, 1.5)
    r = np.random.default_rng(vocab)
    u, k = r.random(rows), r.integers(2100, vocab - 1, rows)
    p = np.where(np.arange(rows) % 2, 1.0, r.uniform(0.05, 0.95, rows))
    k[::4] = 0
    u, p = ([float(np.float32(a)) for a in v] for v in (u, p))
    check(x, u, "searched", k=k.tolist(), p=p)
    d = lambda v, kind: t.tensor(v, dtype=kind, device="cuda")  # noqa: E731
    args = x, d(u, t.float32), None, d(k.tolist(), t.int32), d(p, t.float32)
    first = q.sample(*args)
    for i in range(20):
        say("searched, again", vocab, dtype, i)
        assert t.equal(q.sample(*args), first)


@pytest.mark.parametrize("vocab", [2, 3000, 40007])
def test_numbers_of_one_and_more(vocab):
    """u of 1 and more counts as the largest number below 1, so a last token of less than 2^-24 of the weights is not
    drawn for it."""
    t = torch()
    say("sample: u of 1 and more", vocab)
    x = t.full((6, vocab), -27.0, device="cuda")  # 1.9e-12 each: together less than 2^-24, each more than 2^-42
    x[:, vocab // 2 - 1] = 0.0
    x[5] = 0.0
    u = [1.0, 1.5, float("inf"), 3e38, 0.99999994, 1.0]
    want = [vocab // 2 - 1] * 5 + [vocab - 1]
    for more in ({}, dict(top_k=t.full((6,), vocab, dtype=t.int32, device="cuda")), dict(top_p=t.ones(6, device="cuda")),
                 dict(min_p=t.full((6,), 1e-20, device="cuda"))):
        assert q.sample(x, t.tensor(u, device="cuda"), **more).tolist() == want, more
