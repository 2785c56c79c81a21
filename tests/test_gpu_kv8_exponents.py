"""GPU tests of the cache of 8 bits under every exponent byte that a block may hold, 0 and 255 among them, which count as
1 and 254: what a call leaves of earlier tokens has their values, rounded under the block's new exponent."""
import numpy as np
import pytest

from tests import kv8_ref as ref
from tests.gpu_util import say, torch

pytestmark = pytest.mark.gpu

q = pytest.importorskip("gemm_unpack_bit_amd")

PAGE, DIM = 16, 64
BYTES = [0, 1, 2, 30, 40, 61, 62, 63, 64, 100, 127, 150, 200, 246, 247, 248, 250, 252, 253, 254, 255]


def ints(v):
    return torch().tensor(v, dtype=torch().int32, device="cuda")


def counts_as(e):
    return np.clip(e, 1, 254)


def filled(rows, width, byte_of):
    """A cache of one layer and one head, row b in pages b * width ...; every block's exponents as byte_of gives them
    ([rows, width], keys and values alike), and codes of all kinds.  The cache, its pools, and these on the host."""
    t = torch()
    g = t.Generator(device="cuda").manual_seed(rows)
    pages = rows * width
    codes = [t.randint(0, 256, (1, pages, PAGE, 1, DIM), generator=g, device="cuda", dtype=t.uint8) for _ in range(2)]
    exps = [t.from_numpy(byte_of.astype(np.uint8)).cuda().view(1, pages, 1, 1).clone() for _ in range(2)]
    tables = ints(list(range(pages))).view(rows, width)
    cache = q.KvCache(*[c.view(t.float8_e4m3fn) for c in codes], tables, ints([0] * rows), ints([1] * pages), k_exps=exps[0], v_exps=exps[1])
    host = [ref.Pool(c.cpu().numpy(), counts_as(e.cpu().numpy())) for c, e in zip(codes, exps)]
    return cache, codes, exps, host


def held(codes, exps, host):
    return ref.values(codes.cpu().numpy(), counts_as(exps.cpu().numpy())).reshape(host.v.shape)


@pytest.mark.parametrize("size", ["nothing", "small", "ordinary", "large", "nan"])
def test_append_behind_earlier_tokens(size):
    """Rows of 5 tokens under every byte, and 3 new ones: of zeros, of a size below the least exponent, of ordinary and of
    the largest size, and without a finite value."""
    t = torch()
    say("append8 exponents", size)
    rows = len(BYTES)
    cache, codes, exps, host = filled(rows, 1, np.array(BYTES)[:, None])
    scale = {"nothing": 0.0, "small": 2.0 ** -90, "ordinary": 1.0, "large": 2.0 ** 125, "nan": float("nan")}[size]
    r = np.random.default_rng(3)
    k, v = (t.from_numpy(r.uniform(-1.9, 1.9, (3 * rows, 1, DIM)) * scale).to(t.bfloat16).cuda() for _ in range(2))
    before = [c.clone() for c in codes]
    cu = ints([3 * i for i in range(rows + 1)])
    q.kv_append(cache, 0, k, v, cu, ints([5] * rows))
    for which, x in ((0, k), (1, v)):
        x = x.double().cpu().numpy()
        for b in range(rows):
            host[which].append(0, [b], 5, x[3 * b:3 * b + 3])
        assert np.array_equal(counts_as(exps[which].cpu().numpy()).astype(np.int64).reshape(host[which].e.shape), host[which].e)
        got = held(codes[which], exps[which], host[which]).reshape(rows, PAGE, DIM)
        want = host[which].v.reshape(rows, PAGE, DIM)
        assert np.array_equal(got[:, :8], want[:, :8], equal_nan=True)
        assert t.equal(codes[which][:, :, 8:], before[which][:, :, 8:])


def test_append_in_front_of_nothing():
    """Blocks without earlier tokens take the exponent of the new ones, whatever was there."""
    t = torch()
    say("append8 exponents: empty blocks")
    rows = len(BYTES)
    cache, codes, exps, host = filled(rows, 1, np.array(BYTES)[:, None])
    x = t.randn((rows, 1, DIM), generator=t.Generator(device="cuda").manual_seed(2), device="cuda").bfloat16()
    q.kv_append(cache, 0, x, x, ints(list(range(rows + 1))), ints([0] * rows))
    for b in range(rows):
        host[0].append(0, [b], 0, x[b:b + 1].double().cpu().numpy())
    assert np.array_equal(exps[0].cpu().numpy().astype(np.int64).reshape(host[0].e.shape), host[0].e) and t.equal(exps[0], exps[1])
    got = held(codes[0], exps[0], host[0]).reshape(rows, PAGE, DIM)
    assert np.array_equal(got[:, 0], host[0].v.reshape(rows, PAGE, DIM)[:, 0])


def test_compact_between_blocks():
    """Tokens moved between blocks under every pair of bytes: a block that gains tokens has the largest of the exponents that
    its tokens come from, also where that is below the least that appending gives."""
    t = torch()
    say("kv8_compact exponents")
    pairs = np.array([(a, b) for a in BYTES for b in BYTES])
    rows = len(pairs)
    cache, codes, exps, host = filled(rows, 2, pairs)
    cache.lens.fill_(32)
    # tokens 0 .. 3 stay, then come token 5 and 17, 20 and 31 of the second block
    keep = [1, 13, 16, 27]
    q.kv_compact(cache, ints([4] * rows), ints([keep] * rows), ints([len(keep)] * rows))
    assert int(cache.status) == 0 and cache.lens.tolist() == [4 + len(keep)] * rows
    end = 4 + len(keep)
    for which in range(2):
        for b in range(rows):
            host[which].compact([2 * b, 2 * b + 1], 4, keep)
        got_e = counts_as(exps[which].cpu().numpy()).astype(np.int64).reshape(rows, 2)
        assert np.array_equal(got_e[:, 0], host[which].e.reshape(rows, 2)[:, 0])
        got = held(codes[which], exps[which], host[which]).reshape(rows, 2 * PAGE, DIM)
        assert np.array_equal(got[:, :end], host[which].v.reshape(rows, 2 * PAGE, DIM)[:, :end], equal_nan=True)


def test_compact_takes_the_exponent_of_the_tokens_that_are_left():
    """A block all of whose tokens come from blocks of smaller exponents has theirs afterwards."""
    t = torch()
    say("kv8_compact exponents: all tokens of the block replaced")
    pairs = np.array([(a, b) for a in BYTES for b in BYTES])
    rows = len(pairs)
    cache, codes, exps, host = filled(rows, 2, pairs)
    cache.lens.fill_(32)
    keep = list(range(16, 32))
    q.kv_compact(cache, ints([0] * rows), ints([keep] * rows), ints([16] * rows))
    for which in range(2):
        for b in range(rows):
            host[which].compact([2 * b, 2 * b + 1], 0, keep)
        assert np.array_equal(counts_as(exps[which].cpu().numpy()).astype(np.int64).reshape(rows, 2)[:, 0], counts_as(pairs[:, 1]))
        got = held(codes[which], exps[which], host[which]).reshape(rows, 2 * PAGE, DIM)
        assert np.array_equal(got[:, :16], host[which].v.reshape(rows, 2 * PAGE, DIM)[:, :16], equal_nan=True)


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
def test_read_of_every_code_under_every_byte(dtype):
    """A value read is the cache's, rounded to nearest even where the type does not hold it (below 2^-21 in fp16, below
    2^-130 in bf16), and infinite past the type's range."""
    t = torch()
    say("kv8_read: every code and byte", dtype)
    rows = 256
    cache, codes, exps, _ = filled(rows, 1, np.arange(rows)[:, None])
    for c in codes:
        c.copy_((t.arange(PAGE * DIM, device="cuda") % 256).to(t.uint8).view(1, 1, PAGE, 1, DIM).expand_as(c))
    got = q.kv_read(cache, 0, ints([PAGE * i for i in range(rows + 1)]), ints([0] * rows), tokens=PAGE * rows, dtype=getattr(t, dtype))
    # (exact in 32 bits, subnormal ones too, but for those past 2^128)
    with np.errstate(over="ignore"):
        exact = ref.values(codes[0].cpu().numpy(), counts_as(exps[0].cpu().numpy())).astype(np.float32).reshape(-1, 1, DIM)
    want = t.from_numpy(exact).to(getattr(t, dtype))
    for x in got:
        x = x.cpu()
        same = (x == want) | (x.isnan() & want.isnan())
        assert bool(same.all()), [(float(a), float(b), float(c)) for a, b, c in
                                  zip(x[~same][:9], want[~same][:9], t.from_numpy(exact)[~same][:9])]


@pytest.mark.parametrize("dtype,last", [("float16", 63456.0), ("bfloat16", 247 * 2.0 ** 120)])
def test_the_largest_values_come_back_infinite(dtype, last):
    """The largest code that a type holds is 240 under the exponent of its largest values; from 248 on the nearest is 256."""
    t = torch()
    say("kv8: the largest values", dtype)
    cache, _, _, _ = filled(2, 1, np.full((2, 1), 127))
    x = t.full((2, 1, DIM), last, device="cuda").to(getattr(t, dtype))
    x[1] = 248 * 2.0 ** (8 if dtype == "float16" else 120)
    assert bool(x.isfinite().all()) and float(x[1, 0, 0]) > float(x[0, 0, 0])
    x[1, 0, 1::2] *= -1
    cu = ints([0, 1, 2])
    q.kv_append(cache, 0, x, x, cu, ints([0, 0]))
    for got in q.kv_read(cache, 0, cu, ints([0, 0]), tokens=2, dtype=x.dtype):
        assert bool((got[0] == 240 * 2.0 ** (8 if dtype == "float16" else 120)).all())
        assert bool((got[1, 0, ::2] == float("inf")).all()) and bool((got[1, 0, 1::2] == -float("inf")).all())
