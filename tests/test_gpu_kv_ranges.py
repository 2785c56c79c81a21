"""GPU tests of the cache's calls on row offsets and sizes at the ends of their
ranges: what the device data says must never lead outside the caller's buffers."""
import numpy as np
import pytest

from tests.gpu_util import say, torch

pytestmark = pytest.mark.gpu

q_ = pytest.importorskip("gemm_unpack_bit_amd")


@pytest.mark.parametrize("rows,max_pages", [(1024, 1 << 23), (2100, 1 << 22)])
def test_reserve_adds_up_more_pages_than_32_bits_count(rows, max_pages):
    """Offsets that go up and down ask for up to 2^27 tokens on every second row: together, more pages than 2^31.  The
    rows ask for more than there is, one behind the other; the first one's page is there."""
    t = torch()
    say("kv_reserve far sums", rows, max_pages)
    page, pages = 16, 64
    n = np.full(rows, -1, np.int64)
    n[2::2] = max_pages * page
    n[0] = page
    cu = np.zeros(rows + 1, np.int64)
    up = 0
    for b in range(rows):  # a long row's count is taken back by the short one behind it
        cu[b] = up
        up = up + n[b] if n[b] > 0 else 0
    cu[rows] = up
    count = cu[1:] - cu[:-1]
    assert (count[1::2] < 0).all() and (count[2::2] == max_pages * page).all() and count[0] == page
    assert ((count[count > 0] + page - 1) // page).sum() >= 1 << 31
    free = t.cuda.mem_get_info()[0]
    if free < (rows * max_pages * 4) + (4 << 30):
        pytest.skip("needs a table of 32 GiB")
    tables = t.empty((rows, max_pages), dtype=t.int32, device="cuda")
    tables[:, :3] = -1
    k = t.zeros(1, pages, page, 1, 64, dtype=t.float16, device="cuda")
    zero = lambda m: t.zeros(m, dtype=t.int32, device="cuda")  # noqa: E731
    c = q_.KvCache(k, k.clone(), tables, zero(rows), zero(pages))
    pos = q_.kv_reserve(c, t.from_numpy(cu.astype(np.int32)).cuda())
    assert pos[0] == 0 and bool((pos[1:] == -1).all())
    assert c.lens[0] == page and bool((c.lens[1:] == 0).all())
    assert c.refs.tolist() == [1] + [0] * (pages - 1)
    assert tables[0, :3].tolist() == [0, -1, -1] and bool((tables[1:, :3] == -1).all())
    assert int(c.status) == q_.KV_NO_PAGES | q_.KV_BAD_INDEX


@pytest.mark.parametrize("page", [16, 256])
def test_compact_of_more_tokens_than_the_row_has(page):
    """A count past the row's end at the far end of the longest table: refused, and no position is looked up for it."""
    t = torch()
    say("kv_compact far count", page)
    max_pages = ((1 << 31) - 1024) // page
    cap, keeps = max_pages * page, 4096
    tables = t.zeros((2, max_pages), dtype=t.int32, device="cuda")
    k = t.zeros(1, 4, page, 1, 64, dtype=t.float16, device="cuda")
    refs = t.tensor([1, 1, 1, 1], dtype=t.int32, device="cuda")
    c = q_.KvCache(k, k.clone(), tables, t.tensor([cap, 40], dtype=t.int32, device="cuda"), refs)
    keep = t.arange(keeps, dtype=t.int32, device="cuda").repeat(2, 1)
    pos = t.tensor([cap - 10, 30], dtype=t.int32, device="cuda")
    q_.kv_compact(c, pos, keep, t.tensor([keeps, 11], dtype=t.int32, device="cuda"))
    assert c.lens.tolist() == [cap, 40] and c.refs.tolist() == [1] * 4 and int(c.status) == q_.KV_BAD_INDEX
    assert int(tables.min()) == int(tables.max()) == 0
    c.status.zero_()
    q_.kv_compact(c, pos, keep, t.tensor([10, 10], dtype=t.int32, device="cuda"))  # all that there are: as they lie
    assert c.lens.tolist() == [cap, 40] and int(c.status) == 0
