"""What is measured of the attention and cache operators: cases, their plain forms and their exact values.

Operators: attention over packed prompts (``prompt``), attention of drafted trees or single tokens over a paged
cache (``tree``), growing rows of the cache and writing new keys and values (``append``), forking rows (``fork``)
and keeping a tree's accepted tokens (``compact``).  Head shapes are those of the 8B- and 70B-shaped layers (32 or 64
query heads, 8 key heads, 128 wide), and 64-wide heads.

``run`` computes the plain form (elementary torch operations in 32 bits) or, with ``own`` true, calls the library.
"""
import math
import random

import torch

own = False

DTYPES = {"f16": torch.float16, "bf16": torch.bfloat16}


def _sizes(n, lo, hi):
    """n ragged sizes between lo and hi, spread over their logarithm (the same ones for the same arguments)."""
    return [int(round(lo * (hi / lo) ** ((0.31 + 0.6180339887 * i) % 1.0))) for i in range(n)]


def _cu(sizes):
    out = [0]
    for s in sizes:
        out.append(out[-1] + s)
    return out


def _dev(values, dtype=torch.int32):
    return torch.tensor(values, dtype=dtype, device="cuda")


# ---------------------------------------------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------------------------------------------

def listed():
    return [
        # first turns of a few users, batched: short ragged prompts, where latency counts
        {"name": "prompt_first_turns", "op": "prompt", "heads": 32, "kv": 8, "dim": 128, "dtype": "f16",
         "seqs": 6, "lo": 9, "hi": 300, "past": 0},
        # one long document read at once through a 70B-shaped layer
        {"name": "prompt_one_long", "op": "prompt", "heads": 64, "kv": 8, "dim": 128, "dtype": "f16",
         "seqs": 1, "lo": 16384, "hi": 16384, "past": 0},
        # later turns: new text behind the keys of the earlier ones, 64-wide heads
        {"name": "prompt_later_turns", "op": "prompt", "heads": 32, "kv": 8, "dim": 64, "dtype": "bf16",
         "seqs": 8, "lo": 61, "hi": 1100, "past": 2990},
        # one user, one token: the latency of a decode step
        {"name": "decode_one", "op": "tree", "heads": 32, "kv": 8, "dim": 128, "dtype": "f16",
         "rows": 1, "lo": 777, "hi": 777, "nodes": 1, "page": 16},
        # a decode batch of a 70B-shaped layer over ragged contexts
        {"name": "decode_batch", "op": "tree", "heads": 64, "kv": 8, "dim": 128, "dtype": "f16",
         "rows": 32, "lo": 500, "hi": 16000, "nodes": 1, "page": 16},
        # verification of drafted trees of up to 64 nodes for a batch
        {"name": "tree_batch", "op": "tree", "heads": 32, "kv": 8, "dim": 128, "dtype": "bf16",
         "rows": 16, "lo": 1000, "hi": 8200, "nodes": 64, "page": 64},
        # a decode step's new token of every row
        {"name": "append_decode", "op": "append", "kv": 8, "dim": 128, "dtype": "f16",
         "rows": 48, "lo": 15, "hi": 700, "new_lo": 1, "new_hi": 1, "page": 16},
        # prompts entering the cache
        {"name": "append_prompts", "op": "append", "kv": 8, "dim": 128, "dtype": "f16",
         "rows": 12, "lo": 1, "hi": 90, "new_lo": 100, "new_hi": 3100, "page": 16},
        # a beam search step: every beam goes on from one of the beams before
        {"name": "fork_beams", "op": "fork", "layers": 32, "kv": 8, "dim": 128, "dtype": "f16",
         "rows": 8, "live": 8, "lo": 50, "hi": 400, "page": 16, "wild": True},
        # parallel samples: eight answers from each of four prompts, larger pages
        {"name": "fork_samples", "op": "fork", "layers": 32, "kv": 8, "dim": 128, "dtype": "f16",
         "rows": 32, "live": 4, "lo": 200, "hi": 1500, "page": 64, "wild": False},
        # one user's tree after verification
        {"name": "compact_one", "op": "compact", "layers": 32, "kv": 8, "dim": 128, "dtype": "f16",
         "rows": 1, "lo": 300, "hi": 300, "nodes": 24, "keep": 6, "page": 16},
        # a batch of verified trees
        {"name": "compact_batch", "op": "compact", "layers": 32, "kv": 8, "dim": 128, "dtype": "f16",
         "rows": 48, "lo": 100, "hi": 390, "nodes": 60, "keep": 9, "page": 16},
    ]


def _log(rng, lo, hi):
    return int(round(lo * (hi / lo) ** rng.random()))


def draw(rng):
    op = rng.choice(["prompt", "prompt", "tree", "tree", "append", "fork", "compact"])
    c = {"op": op}
    if op in ("prompt", "tree"):
        c["heads"], c["kv"], c["dim"] = rng.choice([(32, 8, 128), (64, 8, 128), (32, 32, 64), (32, 8, 64), (12, 2, 128),
                                                    (8, 1, 128), (20, 4, 64)])
    else:
        c["kv"], c["dim"] = rng.choice([(8, 128), (8, 64), (2, 128), (1, 128), (32, 64)])
    c["dtype"] = rng.choice(["f16", "bf16"])
    if op == "prompt":
        while True:
            c["seqs"] = _log(rng, 1, 32)
            c["lo"], c["hi"] = sorted((_log(rng, 1, 8192), _log(rng, 1, 8192)))
            c["past"] = rng.choice([0, 0, 0, _log(rng, 1, 16384)])
            if _pairs(c) * c["heads"] * c["dim"] <= 4e11 and c["seqs"] * (c["hi"] + c["past"]) <= 65536:
                return c
    c["page"] = rng.choice([16, 16, 32, 64, 128])
    if op == "tree":
        while True:
            c["rows"] = _log(rng, 1, 64)
            c["lo"], c["hi"] = sorted((_log(rng, 1, 131072), _log(rng, 1, 131072)))
            c["nodes"] = rng.choice([1, 1, _log(rng, 2, 64)])
            keys = sum(_sizes(c["rows"], c["lo"], c["hi"]))
            if keys <= 200000 and keys * c["nodes"] * c["heads"] * c["dim"] <= 6e10:
                return c
    if op == "append":
        while True:
            c["rows"] = _log(rng, 1, 96)
            c["lo"], c["hi"] = sorted((_log(rng, 1, 2000), _log(rng, 1, 2000)))
            c["new_lo"], c["new_hi"] = sorted((_log(rng, 1, 3000), _log(rng, 1, 3000))) if rng.random() < 0.7 else (1, 1)
            if sum(_sizes(c["rows"], c["lo"] + c["new_lo"], c["hi"] + c["new_hi"])) <= 65536:
                return c
    c["layers"] = rng.choice([16, 32, 32])
    if op == "fork":
        while True:
            c["rows"] = _log(rng, 2, 64)
            c["live"] = rng.choice([c["rows"], 1 + rng.randrange(c["rows"])])
            c["lo"], c["hi"] = sorted((_log(rng, 1, 1500), _log(rng, 1, 1500)))
            c["wild"] = rng.random() < 0.6
            if _pool_tokens(c) * c["layers"] * c["kv"] * c["dim"] <= 6e8:
                return c
    while True:
        c["rows"] = _log(rng, 1, 64)
        c["lo"], c["hi"] = sorted((_log(rng, 1, 1500), _log(rng, 1, 1500)))
        c["nodes"] = _log(rng, 2, 64)
        c["keep"] = 1 + rng.randrange(min(c["nodes"], 12))
        if _pool_tokens(c) * c["layers"] * c["kv"] * c["dim"] <= 1e9:
            return c


def _pairs(c):
    """Visible (query, key) pairs of a prompt case."""
    return sum(n * c["past"] + n * (n + 1) // 2 for n in _sizes(c["seqs"], c["lo"], c["hi"]))


def _pool_tokens(c):
    rows = c["rows"] if c["op"] != "fork" else c["live"]
    each = [-(-(s + c.get("nodes", 0)) // c["page"]) for s in _sizes(rows, c["lo"], c["hi"])]
    return (sum(each) + c["rows"] + 8) * c["page"]


def _fork_parents(c):
    """The parent of every new row: any live row (some then die), or each live row's equal share of children."""
    r = random.Random("%d %d %d %d" % (c["rows"], c["live"], c["lo"], c["hi"]))
    return [r.randrange(c["live"]) if c["wild"] else i * c["live"] // c["rows"] for i in range(c["rows"])]


def _kept(c):
    """Per row, the kept nodes in ascending order: the first ones stay in place, the others come from anywhere behind."""
    r = random.Random("%d %d %d %d" % (c["rows"], c["nodes"], c["keep"], c["lo"]))
    out = []
    for b in range(c["rows"]):
        m = c["keep"] if c["rows"] == 1 else r.randint(0, c["keep"])
        still = max(2 * m - c["nodes"], min(m, r.randint(0, 2)))
        out.append(list(range(still)) + sorted(r.sample(range(m, c["nodes"]), m - still)))
    return out


def work(c):
    op, e = c["op"], 2
    if op == "prompt":
        q = _sizes(c["seqs"], c["lo"], c["hi"])
        nq, nk = sum(q), sum(q) + c["past"] * len(q)
        return {"bytes": e * c["dim"] * (2 * nq * c["heads"] + 2 * nk * c["kv"]), "flops": 4 * c["dim"] * c["heads"] * _pairs(c)}
    if op == "tree":
        ctx = _sizes(c["rows"], c["lo"], c["hi"])
        n, keys = c["nodes"] * c["rows"], sum(ctx) + c["nodes"] * c["rows"]
        return {"bytes": e * c["dim"] * (2 * n * c["heads"] + 2 * keys * c["kv"]) + 4 * keys // c["page"],
                "flops": 4 * c["dim"] * c["heads"] * c["nodes"] * (sum(ctx) + c["rows"])}
    if op == "append":
        new = sum(_sizes(c["rows"], c["new_lo"], c["new_hi"]))
        return {"bytes": 2 * 2 * e * new * c["kv"] * c["dim"] + 8 * c["rows"], "flops": 0}
    token = 2 * 2 * e * c["layers"] * c["kv"] * c["dim"]  # one token's keys and values, read and written
    if op == "fork":
        lens, par = _sizes(c["live"], c["lo"], c["hi"]), _fork_parents(c)
        moved = sum(lens[p] % c["page"] for i, p in enumerate(par) if p in par[:i])
        tables = sum(-(-lens[p] // c["page"]) for p in par)
        return {"bytes": token * moved + 8 * tables + 8 * c["rows"], "flops": 0}
    moved = sum(1 for row in _kept(c) for j, s in enumerate(row) if s != j)
    return {"bytes": token * moved + 8 * c["rows"], "flops": 0}


# ---------------------------------------------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------------------------------------------

def _randn(gen, shape, dtype, scale=1.0):
    return torch.randn(shape, generator=gen, device="cuda", dtype=torch.float32).mul_(scale).to(dtype)


def _pool(gen, shape, dtype):
    """A cache's pool: normal values, made in parts to keep the 32-bit draft of them small."""
    out = torch.empty(shape, dtype=dtype, device="cuda")
    for layer in out:
        layer.copy_(torch.randn(layer.shape, generator=gen, device="cuda", dtype=torch.float32))
    return out


def _rows_in_pool(seed, sizes, page, rows, spare_pages, shared=0):
    """Tables and reference counts of `rows` rows, of which the first len(sizes) hold tokens, over shuffled pages; the
    first `shared` pages of every row that has them full are the same ones."""
    r = random.Random(seed)
    need = [-(-s // page) for s in sizes]
    pages = sum(need) + spare_pages
    order = list(range(pages))
    r.shuffle(order)
    width = max(need) + -(-spare_pages // max(1, rows)) + 1
    tables, refs, at = [], [0] * pages, 0
    common = order[len(order) - shared:] if shared else []
    for b in range(rows):
        mine = []
        for i in range(need[b] if b < len(sizes) else 0):
            if i < shared and sizes[b] // page > i:
                mine.append(common[i])
            else:
                mine.append(order[at])
                at += 1
            refs[mine[-1]] += 1
        tables.append(mine + [-1] * (width - len(mine)))
    return tables, refs, pages, width


def _book(tables, lens, refs):
    """One int32 buffer that holds tables, lengths and reference counts, the views into it, and a copy to start from."""
    flat = [p for t in tables for p in t] + lens + refs
    buf = _dev(flat)
    n, m = len(tables) * len(tables[0]), len(lens)
    return buf, buf.clone(), buf[:n].view(len(tables), -1), buf[n:n + m], buf[n + m:]


def _tree_masks(seed, rows, nodes):
    """Ancestor bits of random trees whose nodes follow their parents; node 0 is the root."""
    r = random.Random(seed)
    bits = []
    for _ in range(rows):
        row = []
        for i in range(nodes):
            p = r.randrange(max(0, i - 12), i) if i else None
            row.append((row[p] if i else 0) | 1 << i)
        bits += row
    return [[b - (1 << 64) if b >> 63 else b] for b in bits]


def _inputs(c, seed):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(seed)
    op, dt = c["op"], DTYPES[c["dtype"]]
    if op == "prompt":
        nq = _sizes(c["seqs"], c["lo"], c["hi"])
        nk = [n + c["past"] for n in nq]
        return {"q": _randn(gen, (sum(nq), c["heads"], c["dim"]), dt, 1.5),
                "k": _randn(gen, (sum(nk), c["kv"], c["dim"]), dt),
                "v": _randn(gen, (sum(nk), c["kv"], c["dim"]), dt),
                "nq": nq, "nk": nk, "cu_q": _dev(_cu(nq)), "cu_k": _dev(_cu(nk))}
    if op == "tree":
        ctx = _sizes(c["rows"], c["lo"], c["hi"])
        lens = [n + c["nodes"] for n in ctx]
        tables, refs, pages, _ = _rows_in_pool(seed, lens, c["page"], c["rows"], 8)
        buf, start, t, l, r = _book(tables, lens, refs)
        shape = (1, pages, c["page"], c["kv"], c["dim"])
        return {"q": _randn(gen, (c["rows"] * c["nodes"], c["heads"], c["dim"]), dt, 1.5),
                "k": _pool(gen, shape, dt), "v": _pool(gen, shape, dt), "tables": t, "lens": l, "refs": r,
                "ctx": ctx, "cu": _dev(_cu([c["nodes"]] * c["rows"])), "pos": _dev(ctx),
                "mask": _dev(_tree_masks(seed, c["rows"], c["nodes"]), torch.int64) if c["nodes"] > 1 else None}
    if op == "append":
        lens, new = _sizes(c["rows"], c["lo"], c["hi"]), _sizes(c["rows"], c["new_lo"], c["new_hi"])
        more = sum(-(-(a + b) // c["page"]) - -(-a // c["page"]) for a, b in zip(lens, new))
        tables, refs, pages, width = _rows_in_pool(seed, lens, c["page"], c["rows"], more + 8)
        width = max(-(-(a + b) // c["page"]) for a, b in zip(lens, new))
        tables = [(t + [-1] * width)[:width] for t in tables]
        buf, start, t, l, r = _book(tables, lens, refs)
        shape, T = (1, pages, c["page"], c["kv"], c["dim"]), sum(new)
        # keys and values are parts of a fused product's rows: queries, keys, values
        qkv = _randn(gen, (T, (4 + 2) * c["kv"], c["dim"]), dt)
        return {"k": _pool(gen, shape, dt), "v": _pool(gen, shape, dt), "tables": t, "lens": l, "refs": r, "book": buf,
                "start": start, "cu": _dev(_cu(new)), "new_k": qkv[:, 4 * c["kv"]:5 * c["kv"]],
                "new_v": qkv[:, 5 * c["kv"]:], "total": T}
    if op == "fork":
        lens = _sizes(c["live"], c["lo"], c["hi"])
        tables, refs, pages, _ = _rows_in_pool(seed, lens, c["page"], c["rows"], c["rows"] + 8, shared=2)
        buf, start, t, l, r = _book(tables, lens + [0] * (c["rows"] - c["live"]), refs)
        shape = (c["layers"], pages, c["page"], c["kv"], c["dim"])
        return {"k": _pool(gen, shape, dt), "v": _pool(gen, shape, dt), "tables": t, "lens": l, "refs": r, "book": buf,
                "start": start, "parents": _dev(_fork_parents(c))}
    ctx, kept = _sizes(c["rows"], c["lo"], c["hi"]), _kept(c)
    lens = [n + c["nodes"] for n in ctx]
    tables, refs, pages, _ = _rows_in_pool(seed, lens, c["page"], c["rows"], 8)
    buf, start, t, l, r = _book(tables, lens, refs)
    shape = (c["layers"], pages, c["page"], c["kv"], c["dim"])
    return {"k": _pool(gen, shape, dt), "v": _pool(gen, shape, dt), "tables": t, "lens": l, "refs": r, "book": buf,
            "start": start, "pos": _dev(ctx), "keep": _dev([(k + [-1] * c["keep"])[:c["keep"]] for k in kept]),
            "count": _dev([len(k) for k in kept])}


def prepare(case, seed):
    s = _inputs(case, seed)
    s["case"] = case
    if own:
        import gemm_unpack_bit_amd as q

        op = case["op"]
        if op != "prompt":
            s["cache"] = q.KvCache(s["k"], s["v"], s["tables"], s["lens"], s["refs"])
        if op == "prompt":
            n = q.attn_prompt_workspace_bytes(s["q"].shape[0], s["k"].shape[0], case["seqs"], case["heads"], case["kv"],
                                              case["dim"])
        elif op == "tree":
            n = q.attn_tree_workspace_bytes(s["q"].shape[0], case["rows"], case["heads"], case["kv"], case["dim"])
        if op in ("prompt", "tree"):
            s["ws"] = torch.empty(max(n, 16), dtype=torch.uint8, device="cuda")
            s["out"] = torch.empty_like(s["q"])
        if op == "append":
            s["pos"] = torch.empty(case["rows"], dtype=torch.int32, device="cuda")
        if op == "fork":
            s["forked"] = s["cache"].empty_rows()
    return s


# ---------------------------------------------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------------------------------------------

def run(s):
    return (_run_own if own else _run_plain)[s["case"]["op"]](s)


def _own_prompt(s):
    import gemm_unpack_bit_amd as q

    return q.attn_prompt(s["q"], s["k"], s["v"], s["cu_q"], s["cu_k"], out=s["out"], ws=s["ws"])


def _own_tree(s):
    import gemm_unpack_bit_amd as q

    return q.attn_tree(s["q"], s["cache"], 0, s["cu"], s["pos"], s["mask"], out=s["out"], ws=s["ws"])


def _own_append(s):
    import gemm_unpack_bit_amd as q

    s["book"].copy_(s["start"])  # every pass grows the same rows
    q.kv_reserve(s["cache"], s["cu"], out=s["pos"])
    q.kv_write(s["cache"], 0, s["new_k"], s["new_v"], s["cu"], s["pos"])
    return [s["k"], s["v"], s["tables"], s["lens"], s["refs"], s["pos"]]


def _own_fork(s):
    import gemm_unpack_bit_amd as q

    s["book"].copy_(s["start"])
    f = q.kv_fork(s["cache"], s["parents"], out=s["forked"])
    return [s["k"], s["v"], f.tables, f.lens, s["refs"]]


def _own_compact(s):
    import gemm_unpack_bit_amd as q

    s["book"].copy_(s["start"])
    q.kv_compact(s["cache"], s["pos"], s["keep"], s["count"])
    return [s["k"], s["v"], s["tables"], s["lens"], s["refs"]]


_run_own = {"prompt": _own_prompt, "tree": _own_tree, "append": _own_append, "fork": _own_fork, "compact": _own_compact}


def _softmax_rows(scores, visible):
    """Weights of the visible scores of each row and their sum; a row without any has weights 0 and sum 1."""
    m = scores.masked_fill(~visible, -math.inf).amax(-1, keepdim=True)
    m = torch.where(m == -math.inf, torch.zeros_like(m), m)
    p = torch.where(visible, torch.exp(scores - m), torch.zeros_like(scores))
    total = p.sum(-1, keepdim=True)
    return p, torch.where(total == 0, torch.ones_like(total), total)


def _plain_prompt(s, step=2048):
    c, q, k, v = s["case"], s["q"], s["k"], s["v"]
    out, group, scale = torch.empty_like(q), c["heads"] // c["kv"], 1.0 / math.sqrt(c["dim"])
    q0 = k0 = 0
    for nq, nk in zip(s["nq"], s["nk"]):
        cols = torch.arange(nk, device="cuda")
        for h in range(c["kv"]):
            kt = k[k0:k0 + nk, h].float().t().contiguous()
            vh = v[k0:k0 + nk, h].float()
            for a in range(0, nq, step):
                b = min(nq, a + step)
                qh = q[q0 + a:q0 + b, h * group:(h + 1) * group].float().transpose(0, 1).reshape(-1, c["dim"])
                rows = torch.arange(a, b, device="cuda").repeat(group)
                p, total = _softmax_rows((qh @ kt) * scale, cols[None, :] <= nk - nq + rows[:, None])
                o = ((p @ vh) / total).view(group, b - a, c["dim"]).transpose(0, 1)
                out[q0 + a:q0 + b, h * group:(h + 1) * group] = o.to(q.dtype)
        q0, k0 = q0 + nq, k0 + nk
    return out


def _plain_tree(s):
    c, q = s["case"], s["q"]
    n, group, scale = c["nodes"], c["heads"] // c["kv"], 1.0 / math.sqrt(c["dim"])
    out = torch.empty_like(q)
    nodes = torch.arange(n, device="cuda")
    for b, ctx in enumerate(s["ctx"]):
        t = s["tables"][b, :-(-(ctx + n) // c["page"])].long()
        k = s["k"][0][t].reshape(-1, c["kv"], c["dim"])[:ctx + n].float().permute(1, 2, 0).contiguous()
        v = s["v"][0][t].reshape(-1, c["kv"], c["dim"])[:ctx + n].float().transpose(0, 1).contiguous()
        qh = q[b * n:(b + 1) * n].float().view(n, c["kv"], group, c["dim"]).permute(1, 2, 0, 3).reshape(c["kv"], -1, c["dim"])
        visible = torch.ones((n, ctx + n), dtype=torch.bool, device="cuda")
        if s["mask"] is not None:
            visible[:, ctx:] = ((s["mask"][b * n:(b + 1) * n] >> nodes[None, :]) & 1) != 0
        p, total = _softmax_rows((qh @ k) * scale, visible.repeat(group, 1)[None])
        o = ((p @ v) / total).view(c["kv"], group, n, c["dim"]).permute(2, 0, 1, 3)
        out[b * n:(b + 1) * n] = o.reshape(n, c["heads"], c["dim"]).to(q.dtype)
    return out


def _plain_append(s):
    c, page = s["case"], s["case"]["page"]
    s["book"].copy_(s["start"])
    tables, lens, refs, cu = s["tables"], s["lens"], s["refs"], s["cu"].long()
    add = cu[1:] - cu[:-1]
    pos = lens.clone()
    have, want = (pos.long() + page - 1) // page, (pos.long() + add + page - 1) // page
    slots = torch.arange(tables.shape[1], device="cuda")[None, :]
    fresh = (slots >= have[:, None]) & (slots < want[:, None])
    free = (refs == 0).nonzero()[:, 0]  # lowest numbers first
    rank = (torch.cumsum(fresh.reshape(-1).long(), 0) - 1).view_as(fresh).clamp(min=0)
    tables.copy_(torch.where(fresh, free[rank.clamp(max=free.numel() - 1)].int(), tables))
    refs[tables[fresh].long()] = 1
    lens.add_(add.int())
    token = torch.arange(s["total"], device="cuda")
    row = torch.searchsorted(cu[1:].contiguous(), token, right=True)
    at = pos[row].long() + token - cu[row]
    where = tables[row, at // page].long() * page + at % page
    s["k"].view(-1, c["kv"], c["dim"])[where] = s["new_k"]
    s["v"].view(-1, c["kv"], c["dim"])[where] = s["new_v"]
    return [s["k"], s["v"], tables, lens, refs, pos]


def _plain_fork(s):
    page, par = s["case"]["page"], s["parents"].long()
    s["book"].copy_(s["start"])
    tables, lens, refs = s["tables"], s["lens"].long(), s["refs"]
    n = par.numel()
    ids = torch.arange(n, device="cuda")
    same = par[:, None] == par[None, :]
    first = ~(same & (ids[None, :] < ids[:, None])).any(1)
    children = (par[None, :] == ids[:, None]).sum(1)
    slots = torch.arange(tables.shape[1], device="cuda")[None, :]
    full, part = lens // page, lens % page
    delta = torch.where(slots < full[:, None], children[:, None] - 1, torch.zeros_like(slots))
    tail = (slots == full[:, None]) & (part > 0)[:, None]
    delta = torch.where(tail & (children == 0)[:, None], torch.full_like(delta, -1), delta)
    refs.index_add_(0, tables.clamp(min=0).reshape(-1), delta.reshape(-1).int())
    copy = (part[par] > 0) & ~first
    free = (refs == 0).nonzero()[:, 0]
    fresh = free[(torch.cumsum(copy.long(), 0) - 1).clamp(min=0)]
    new_lens = lens[par]
    new = torch.where(slots < full[par][:, None] + (part[par] > 0)[:, None].long(), tables[par], torch.full_like(tables, -1))
    new = torch.where(copy[:, None] & (slots == full[par][:, None]), fresh[:, None].int(), new)
    old = tables[par, full[par].clamp(max=tables.shape[1] - 1)].long()
    who = copy.nonzero()[:, 0]
    refs[fresh[who]] = 1
    held = torch.arange(page, device="cuda")[None, :] < part[par][who][:, None]
    for pool in (s["k"], s["v"]):
        for layer in pool:
            layer[fresh[who]] = torch.where(held[..., None, None], layer[old[who]], layer[fresh[who]])
    return [s["k"], s["v"], new, new_lens.int(), refs]


def _plain_compact(s):
    c, page = s["case"], s["case"]["page"]
    s["book"].copy_(s["start"])
    tables, lens, refs, pos = s["tables"], s["lens"], s["refs"], s["pos"].long()
    j = torch.arange(c["keep"], device="cuda")[None, :]
    keep, count = s["keep"].long(), s["count"].long()
    src, dst = pos[:, None] + keep.clamp(min=0), pos[:, None] + j
    move = (j < count[:, None]) & (src != dst)
    src = tables.gather(1, src // page).long() * page + src % page
    dst = tables.gather(1, (dst // page).clamp(max=tables.shape[1] - 1)).long() * page + dst % page
    src, dst = src[move], dst[move]
    for pool in (s["k"], s["v"]):
        flat = pool.view(c["layers"], -1, c["kv"], c["dim"])
        flat[:, dst] = flat[:, src]
    have, want = (lens.long() + page - 1) // page, (pos + count + page - 1) // page
    slots = torch.arange(tables.shape[1], device="cuda")[None, :]
    gone = (slots >= want[:, None]) & (slots < have[:, None])
    refs.index_add_(0, tables.clamp(min=0).reshape(-1), torch.where(gone, -1, 0).reshape(-1).int())
    tables.masked_fill_(gone, -1)
    lens.copy_((pos + count).int())
    return [s["k"], s["v"], tables, lens, refs]


_run_plain = {"prompt": _plain_prompt, "tree": _plain_tree, "append": _plain_append, "fork": _plain_fork,
              "compact": _plain_compact}


# ---------------------------------------------------------------------------------------------------------------
# exact values: attention from its definition in 64 bits, head by head; the cache's state row by row on the host
# ---------------------------------------------------------------------------------------------------------------

def _attend(q, k, v, seen, scale):
    """softmax(q k^T) v over the keys that `seen` marks, in 64 bits: q [n, D], k and v [m, D], seen [n, m]."""
    logits = (q.double() * scale).matmul(k.double().t().contiguous())
    logits[~seen] = -math.inf
    none = ~seen.any(1)
    logits[none] = 0.0
    out = torch.exp(logits - torch.logsumexp(logits, 1, keepdim=True)).matmul(v.double())
    out[none] = 0.0
    return out


def exact(case, seed):
    s = _inputs(case, seed)
    op = case["op"]
    if op in ("prompt", "tree"):
        q, per, scale = s["q"], case["heads"] // case["kv"], case["dim"] ** -0.5
        out = torch.zeros(q.shape, dtype=torch.float64, device="cuda")
        if op == "prompt":
            at_q = at_k = 0
            for nq, nk in zip(s["nq"], s["nk"]):
                where = torch.arange(nk, device="cuda")
                for a in range(0, nq, 4096):
                    i = torch.arange(a, min(nq, a + 4096), device="cuda") + (nk - nq)
                    seen = where.unsqueeze(0) <= i.unsqueeze(1)
                    for h in range(case["heads"]):
                        rows = slice(at_q + a, at_q + a + i.numel())
                        out[rows, h] = _attend(q[rows, h], s["k"][at_k:at_k + nk, h // per], s["v"][at_k:at_k + nk, h // per],
                                               seen, scale)
                at_q, at_k = at_q + nq, at_k + nk
            return out
        n, tables = case["nodes"], s["tables"].tolist()
        masks = s["mask"].view(-1).tolist() if s["mask"] is not None else [1] * q.shape[0]
        for b, ctx in enumerate(s["ctx"]):
            order = torch.tensor([tables[b][p // case["page"]] * case["page"] + p % case["page"] for p in range(ctx + n)],
                                 device="cuda")
            seen = torch.tensor([[(masks[b * n + i] >> j) & 1 == 1 for j in range(n)] for i in range(n)], device="cuda")
            seen = torch.cat([torch.ones((n, ctx), dtype=torch.bool, device="cuda"), seen], 1)
            for h in range(case["heads"]):
                kk = s["k"].view(-1, case["kv"], case["dim"])[order, h // per]
                vv = s["v"].view(-1, case["kv"], case["dim"])[order, h // per]
                out[b * n:(b + 1) * n, h] = _attend(q[b * n:(b + 1) * n, h], kk, vv, seen, scale)
        return out
    page, tables, lens, refs = case["page"], s["tables"].tolist(), s["lens"].tolist(), s["refs"].tolist()
    src, dst = [], []  # token places in the pool, moved from the state before
    if op == "append":
        pos, cu = list(lens), s["cu"].tolist()
        for b in range(case["rows"]):
            for i in range(cu[b], cu[b + 1]):
                if lens[b] % page == 0:
                    got = refs.index(0)
                    refs[got], tables[b][lens[b] // page] = 1, got
                dst.append(tables[b][lens[b] // page] * page + lens[b] % page)
                lens[b] += 1
        for pool, new in ((s["k"], s["new_k"]), (s["v"], s["new_v"])):
            pool.view(-1, case["kv"], case["dim"]).index_copy_(0, _dev(dst, torch.int64), new.contiguous())
        return [s["k"], s["v"], _dev(tables), _dev(lens), _dev(refs), _dev(pos)]
    if op == "fork":
        par, width = s["parents"].tolist(), len(tables[0])
        for p in range(case["rows"]):
            for i in range(-(-lens[p] // page)):
                whole = (i + 1) * page <= lens[p]
                refs[tables[p][i]] += par.count(p) - 1 if whole else min(0, par.count(p) - 1)
        rows = []
        for i, p in enumerate(par):
            row = list(tables[p][:-(-lens[p] // page)])
            if lens[p] % page and p in par[:i]:
                got = refs.index(0)
                refs[got] = 1
                src += [row[-1] * page + t for t in range(lens[p] % page)]
                dst += [got * page + t for t in range(lens[p] % page)]
                row[-1] = got
            rows.append(row + [-1] * (width - len(row)))
        tables, lens = rows, [lens[p] for p in par]
    else:
        for b, (pos, kept) in enumerate(zip(s["pos"].tolist(), _kept(case))):
            for j, i in enumerate(kept):
                src.append(tables[b][(pos + i) // page] * page + (pos + i) % page)
                dst.append(tables[b][(pos + j) // page] * page + (pos + j) % page)
            for i in range(-(-(pos + len(kept)) // page), -(-lens[b] // page)):
                refs[tables[b][i]] -= 1
                tables[b][i] = -1
            lens[b] = pos + len(kept)
    if src:
        a, b = _dev(src, torch.int64), _dev(dst, torch.int64)
        for pool in (s["k"], s["v"]):
            for layer in pool.view(case["layers"], -1, case["kv"] * case["dim"]):
                layer.index_copy_(0, b, layer.index_select(0, a))
    return [s["k"], s["v"], _dev(tables), _dev(lens), _dev(refs)]
