"""GPU tests of layouts that a user's arrays come in and the other tests do not have."""
import pytest

from tests.gpu_util import say, torch

pytestmark = pytest.mark.gpu

q_ = pytest.importorskip("gemm_unpack_bit_amd")


@pytest.mark.parametrize("dtype", ["float16", "bfloat16"])
@pytest.mark.parametrize("H,KV,D", [(8, 2, 128), (4, 4, 64)])
def test_one_token_of_a_padded_row(dtype, H, KV, D):
    """A single token's row stride is whatever its buffer's was (``contiguous`` leaves such a view alone)."""
    t = torch()
    say("attention strides of one", dtype, H, KV, D)
    dt, g = getattr(t, dtype), t.Generator(device="cuda").manual_seed(3)
    padded = lambda x, n: x[:, :n * D].view(3, n, D)[:1]  # noqa: E731 (the first of three rows)
    row = padded(t.randn(3, (H + 2 * KV) * D + 4, generator=g, device="cuda").to(dt), H + 2 * KV)
    assert row.stride(0) % 8 and row.is_contiguous()
    plain = row.clone(memory_format=t.contiguous_format).view(-1).clone().view(1, H + 2 * KV, D)
    assert plain.stride(0) % 8 == 0
    cu = t.tensor([0, 1], dtype=t.int32, device="cuda")
    split = lambda x: (x[:, :H], x[:, H:H + KV], x[:, H + KV:])  # noqa: E731
    (q, k, v), (q2, k2, v2) = split(row), split(plain)
    out = t.full((3, H * D + 4), 7.0, dtype=dt, device="cuda")
    o = q_.attn_prompt(q, k, v, cu, out=padded(out, H))
    assert t.equal(o, q_.attn_prompt(q2, k2, v2, cu)) and bool((out[:, H * D:] == 7).all()) and bool((out[1:] == 7).all())
    assert t.equal(o, v.repeat_interleave(H // KV, 1))  # the one key
    caches = []
    for kk, vv, qq in ((k, v, q), (k2, v2, q2)):
        c = q_.KvCache.empty(1, 4, 16, KV, D, 1, 2, dtype=dt)
        c.k.zero_(), c.v.zero_()
        pos = q_.kv_reserve(c, cu)
        q_.kv_write(c, 0, kk, vv, cu, pos)
        caches.append((c.k, c.v, q_.attn_tree(qq, c, 0, cu, pos)))
    for a, b in zip(*caches):
        assert t.equal(a, b)
    assert t.equal(caches[0][2], o)


@pytest.mark.parametrize("n", [5, 200])
def test_one_head_of_a_wider_array(n):
    t = torch()
    say("attention head stride of one head", n)
    g = t.Generator(device="cuda").manual_seed(4)
    x = [t.randn(2, n * 64 + 4, generator=g, device="cuda").half()[:, :n * 64].view(2, n, 64)[:1].transpose(0, 1) for _ in range(3)]
    assert x[0].stride(1) % 8
    cu = t.tensor([0, n], dtype=t.int32, device="cuda")
    assert t.equal(q_.attn_prompt(*x, cu), q_.attn_prompt(*(y.reshape(-1).clone().view(n, 1, 64) for y in x), cu))
