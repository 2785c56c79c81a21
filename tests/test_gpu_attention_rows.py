"""GPU parity of the attention calls where their work is split: prompts whose keys
are cut over workgroups, and batches of more rows than a wave has lanes, in every
kernel; rows of unlike length, empty ones among them."""
import numpy as np
import pytest

from tests.gpu_util import say, torch
from tests.test_gpu_attention import _cache, _check_prompt, _check_tree, _cu, _dt, _gen, _rand, _tree, _words

pytestmark = pytest.mark.gpu

q_ = pytest.importorskip("gemm_unpack_bit_amd")


def _is_wide(tokens, rows, group):
    return -(-tokens // rows) * group > 32


SPLIT = [
    # (nq, nk): more than 2048 keys a sequence on average, few query tiles
    ([70], [2100]),
    ([300], [9000]),
    ([150, 130], [6000, 2500]),
    ([90, 0, 400, 65], [30, 5000, 12000, 64]),  # one with fewer keys than queries, one without queries
    ([129, 200], [0, 8192]),                    # one without keys
]


@pytest.mark.parametrize("dtype", ["f16", "bf16"])
@pytest.mark.parametrize("heads,kv,D", [(4, 1, 128), (4, 4, 64), (6, 2, 64), (3, 3, 128)])
@pytest.mark.parametrize("case", range(len(SPLIT)))
@pytest.mark.parametrize("causal", [True, False])
def test_prompts_whose_keys_are_split(dtype, heads, kv, D, case, causal):
    nq, nk = SPLIT[case]
    say("attn_prompt split", dtype, heads, kv, D, nq, nk, causal)
    t, g, dt = torch(), _gen(case + 100), _dt(dtype)
    assert _is_wide(sum(nq), len(nq), heads // kv)
    # (the wide kernel has a workspace only where it splits the keys)
    assert q_.attn_prompt_workspace_bytes(sum(nq), sum(nk), len(nq), heads, kv, D) > 0
    q = _rand(g, sum(nq), heads, D, dtype=dt, scale=2.0)
    k, v = _rand(g, sum(nk), kv, D, dtype=dt), _rand(g, sum(nk), kv, D, dtype=dt)
    out = t.full_like(q, float("nan"))
    q_.attn_prompt(q, k, v, _cu(nq), _cu(nk), causal=causal, out=out)
    _check_prompt(out, q, k, v, nq, nk, causal, D ** -0.5, dtype, f"split {nq} {nk}", most=24)
    assert t.equal(out, q_.attn_prompt(q, k, v, _cu(nq), _cu(nk), causal=causal)), "not deterministic"


def _ragged(rng, rows, most, long_at, long):
    n = rng.integers(0, most + 1, rows).tolist()
    n[0], n[rows // 2], n[-1] = 0, 0, 1
    n[long_at] = long
    return n


@pytest.mark.parametrize("rows", [65, 130, 300])
@pytest.mark.parametrize("heads,kv,D,dtype", [(16, 1, 128, "f16"), (32, 2, 64, "bf16")])
@pytest.mark.parametrize("causal", [True, False])
def test_wide_prompts_of_many_sequences(rows, heads, kv, D, dtype, causal):
    say("attn_prompt many wide", rows, heads, kv, D, dtype, causal)
    rng, g, dt = np.random.default_rng(rows), _gen(rows), _dt(dtype)
    nq = _ragged(rng, rows, 9, 64, 333)
    nk = [n + int(rng.integers(0, 60)) for n in nq]
    nk[5] = 0
    assert _is_wide(sum(nq), rows, heads // kv)
    q = _rand(g, sum(nq), heads, D, dtype=dt, scale=2.0)
    k, v = _rand(g, sum(nk), kv, D, dtype=dt), _rand(g, sum(nk), kv, D, dtype=dt)
    out = q_.attn_prompt(q, k, v, _cu(nq), _cu(nk), causal=causal)
    _check_prompt(out, q, k, v, nq, nk, causal, D ** -0.5, dtype, f"{rows} sequences", most=20)


@pytest.mark.parametrize("D,dtype", [(128, "bf16"), (64, "f16")])
def test_split_prompts_of_many_sequences(D, dtype):
    rows, heads = 70, 16
    say("attn_prompt many split", D, dtype)
    rng, g, dt = np.random.default_rng(7), _gen(7), _dt(dtype)
    nq = _ragged(rng, rows, 6, 66, 40)
    nk = rng.integers(0, 4400, rows).tolist()
    nk[66] = 9000
    assert _is_wide(sum(nq), rows, heads) and q_.attn_prompt_workspace_bytes(sum(nq), sum(nk), rows, heads, 1, D) > 0
    q = _rand(g, sum(nq), heads, D, dtype=dt, scale=2.0)
    k, v = _rand(g, sum(nk), 1, D, dtype=dt), _rand(g, sum(nk), 1, D, dtype=dt)
    _check_prompt(q_.attn_prompt(q, k, v, _cu(nq), _cu(nk)), q, k, v, nq, nk, True, D ** -0.5, dtype, "many split", most=8)


@pytest.mark.parametrize("rows", [65, 130, 300])
@pytest.mark.parametrize("heads,kv,D,dtype,kernel", [
    (4, 2, 128, "bf16", "narrow"), (6, 1, 64, "f16", "narrow"),           # up to 16 and 32 query rows a key head
    (16, 1, 128, "f16", "wide"), (32, 2, 64, "bf16", "wide"),             # four waves
    (64, 2, 128, "bf16", "wide"), (32, 1, 64, "f16", "wide"),             # eight
])
@pytest.mark.parametrize("drafted", [False, True])
def test_trees_of_many_rows(rows, heads, kv, D, dtype, kernel, drafted):
    """One row is long enough for its parts to lie in many workgroups, and stands where the rows' second 64 begin."""
    say("attn_tree many rows", rows, heads, kv, D, dtype, kernel, drafted)
    rng, dt = np.random.default_rng(rows + heads), _dt(dtype)
    ns = _ragged(rng, rows, 9, 64, 20)
    pos = rng.integers(0, 150, rows).tolist()
    pos[64], pos[63], pos[7] = 9000, 3000, -1
    group, mean = heads // kv, -(-sum(ns) // rows)
    assert (kernel == "wide") == _is_wide(sum(ns), rows, group) and (mean * group > 128) == (group == 32)
    cache, tables = _cache(rows, dt, [max(p, 0) + n if p >= 0 else 9 for p, n in zip(pos, ns)], 32, kv, D, fill=float("nan"))
    q = _rand(_gen(rows), sum(ns), heads, D, dtype=dt, scale=2.0)
    p = torch().tensor(pos, dtype=torch().int32, device="cuda")
    bits = [b for n in ns for b in _tree(rng, n)] if drafted else None
    mask = _words(bits, 1) if drafted else None
    out = torch().full_like(q, float("nan"))
    q_.attn_tree(q, cache, 0, _cu(ns), p, mask, out=out)
    _check_tree(out, q, cache, 0, tables, ns, pos, bits, D ** -0.5, dtype, f"{rows} rows", most=20)
    assert torch().equal(out, q_.attn_tree(q, cache, 0, _cu(ns), p, mask)), "not deterministic"


def test_a_long_row_between_many_short_ones():
    """Two rows of one key head, one long: as many parts of it as there are workgroups, all joined."""
    say("attn_tree skewed")
    ns, pos = [1, 1], [150000, 0]
    cache, tables = _cache(5, _dt("f16"), [150001, 1], 256, 1, 64, fill=float("nan"))
    q = _rand(_gen(5), 2, 4, 64, dtype=_dt("f16"), scale=2.0)
    p = torch().tensor(pos, dtype=torch().int32, device="cuda")
    _check_tree(q_.attn_tree(q, cache, 0, _cu(ns), p), q, cache, 0, tables, ns, pos, None, 0.125, "f16", "skewed")
