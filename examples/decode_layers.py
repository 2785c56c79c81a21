"""Prompts, forked rows, drafted trees and decode steps through a small stack of decoder layers.

    python examples/decode_layers.py

The weights are random 4-bit codes, so what the tokens say means nothing; the
calls and their order are those of a serving loop:

- prompts      kv_reserve once, then per layer rms_norm, kv_append (rotation and
               the cache in one), kv_read and attn_prompt;
- a decode step  the same with attn_tree over the cache, one token per row, and
               sample (here the largest logit) at its end;
- scouting     kv_fork gives every row a twin that decodes a few tokens ahead,
               and a second kv_fork drops the twins (their pages go back);
- verification attn_tree over each row's drafted tree (the scouted tokens and
               wrong guesses beside them), every node seeing its ancestors;
- acceptance   kv_compact keeps the nodes that the layers agree with.

The cache is of 16 bits, or with ``main(cache_type=torch.float8_e4m3fn)`` of 8.
At the end the next token's logits over the cache are compared with those of
one prompt that holds all the kept tokens.
"""
from __future__ import annotations

import math
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import gemm_unpack_bit_amd as q  # noqa: E402

LAYERS, HIDDEN, HEADS, HEADS_KV, DIM, FFN, VOCAB, BITS = 2, 512, 8, 2, 64, 1024, 1024, 4
PAGE = 16


class Linear:
    """A product with packed 4-bit weights: the decode kernels up to 16 rows, the prompt kernel above."""

    def __init__(self, gen, n, k):
        codes = torch.randint(0, 16, (n, k), generator=gen, device="cuda", dtype=torch.uint8)
        zeros = torch.randint(0, 16, (n, k // 128), generator=gen, device="cuda", dtype=torch.uint8)
        self.wq, self.zeros = q.pack(codes, BITS), q.pack_zeros(zeros, BITS)
        # codes minus zero points have a deviation of about 6.5: outputs about as large as inputs
        self.scales = (torch.rand(n, k // 128, generator=gen, device="cuda") + 0.5).mul_(1 / (6.5 * math.sqrt(k))).half()

    def __call__(self, x):
        f = q.uniform if x.shape[0] <= 16 else q.gemm_uniform
        return f(x.contiguous(), self.wq, self.scales, self.zeros, BITS)


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def offsets(counts):
    out = [0]
    for n in counts:
        out.append(out[-1] + n)
    return ints(out)


class Model:
    def __init__(self, seed):
        gen = torch.Generator(device="cuda")
        gen.manual_seed(seed)
        self.embed = torch.randn(VOCAB, HIDDEN, generator=gen, device="cuda").half()
        self.layers = [dict(qkv=Linear(gen, (HEADS + 2 * HEADS_KV) * DIM, HIDDEN), out=Linear(gen, HIDDEN, HEADS * DIM),
                            up=Linear(gen, 2 * FFN, HIDDEN), down=Linear(gen, HIDDEN, FFN)) for _ in range(LAYERS)]
        self.head = Linear(gen, VOCAB, HIDDEN)
        self.weight = torch.ones(HIDDEN, device="cuda").half()  # of every norm
        self.freqs = 10000.0 ** (-torch.arange(DIM // 2, device="cuda") / (DIM // 2))

    def run(self, tokens, at, cache, cu, mask=None, prompt=False):
        """Logits of ``tokens`` (packed rows, ``cu``) at the positions ``at`` (int32); the rows of the cache grow by them.
        Returns the logits and where each row's tokens begin in its row."""
        x, more = self.embed[tokens], None  # the sum so far, and what the last product adds to it
        pos = q.kv_reserve(cache, cu)

        def norm():
            if more is None:
                return q.rms_norm(x, self.weight), x
            return q.rms_norm(more, self.weight, residual=x, residual_out=x)

        for n, layer in enumerate(self.layers):
            y, x = norm()
            qkv = layer["qkv"](y).view(-1, HEADS + 2 * HEADS_KV, DIM)
            qh, kh, vh = qkv.split([HEADS, HEADS_KV, HEADS_KV], 1)  # views: their token stride is the product's row
            q.kv_append(cache, n, kh, vh, cu, pos, q=qh, freqs=self.freqs, at=at, out=qh)
            if prompt:
                kh, vh = q.kv_read(cache, n, cu, pos, tokens=len(tokens))
                o = q.attn_prompt(qh, kh, vh, cu)
            else:
                o = q.attn_tree(qh, cache, n, cu, pos, mask)
            more = layer["out"](o.view(-1, HEADS * DIM))
            y, x = norm()
            gate, up = layer["up"](y).chunk(2, -1)
            more = layer["down"](torch.nn.functional.silu(gate) * up)
        return self.head(norm()[0]), pos

    def prompts(self, texts, cache):
        at = torch.cat([torch.arange(len(t), dtype=torch.int32, device="cuda") for t in texts])
        cu = offsets([len(t) for t in texts])
        logits, _ = self.run(torch.cat(texts), at, cache, cu, prompt=True)
        return logits[cu[1:].long() - 1]

    def step(self, tokens, cache):
        return self.run(tokens, cache.lens.clone(), cache, offsets([1] * cache.rows))[0]


def new_cache(rows, kind):
    return q.KvCache.empty(LAYERS, 64, PAGE, HEADS_KV, DIM, rows, 24, dtype=kind)


def largest(logits):
    """The tokens that sampling at a temperature of 0 takes."""
    none = torch.zeros(len(logits), device="cuda")
    return q.sample(logits, none, temperature=none).long()


def tree_of(chain, gen):
    """A drafted tree: the row's pending token, the scouted ones as a path below it, and a wrong guess beside each.
    Returns tokens, parents (-1: the root), in an order in which a parent stands before its children."""
    tokens, parents, last = [chain[0]], [-1], 0
    for t in chain[1:]:
        guess = int(torch.randint(0, VOCAB, (1,), generator=gen))
        tokens += [guess if guess != t else (t + 1) % VOCAB, t]
        parents += [last, last]
        last = len(tokens) - 1
    return tokens, parents


def main(seed=1, lengths=(37, 5, 120), ahead=4, rounds=2, cache_type=torch.float16):
    model, gen = Model(seed), torch.Generator().manual_seed(seed)
    texts = [torch.randint(0, VOCAB, (n,), generator=gen).cuda() for n in lengths]
    rows = len(texts)
    cache = new_cache(rows, cache_type)
    pending = largest(model.prompts(texts, cache))  # of every row: chosen, not in the cache yet
    accepted = []
    for _ in range(rounds):
        # scout: twins decode `ahead` tokens, then their rows end
        twins = q.kv_fork(cache, ints([b for b in range(rows) for _ in range(2)]))
        chains, t = [[int(p)] for p in pending], pending.repeat_interleave(2)
        idle = ints([0] * (2 * rows))
        for _ in range(ahead):
            logits = model.step(t, twins)
            t = largest(logits).view(rows, 2)[:, :1].repeat(1, 2).flatten()
            for b in range(rows):
                chains[b].append(int(t[2 * b]))
        # the twin at 2 b + 1 goes back to where the row was (it stepped along), the scout at 2 b ends
        q.kv_compact(twins, twins.lens - ahead, idle.view(-1, 1), idle)
        cache = q.kv_fork(twins, ints([2 * b + 1 for b in range(rows)]))
        # verify all trees at once
        trees = [tree_of(c, gen) for c in chains]
        tokens, at, mask, lens = [], [], [], cache.lens.tolist()
        for b, (tok, par) in enumerate(trees):
            seen, depth = [], []
            for i, p in enumerate(par):
                seen.append((seen[p] if p >= 0 else 0) | 1 << i)
                depth.append(depth[p] + 1 if p >= 0 else 0)
            tokens += tok
            at += [lens[b] + d for d in depth]
            mask += [[s] for s in seen]
        cu = offsets([len(tok) for tok, _ in trees])
        logits, pos = model.run(torch.tensor(tokens, device="cuda"), ints(at), cache, cu,
                                torch.tensor(mask, device="cuda"))
        best, first = largest(logits).tolist(), cu.tolist()
        # accept from each root on, as long as a child is what the layers would say next
        keep = []
        for b, (tok, par) in enumerate(trees):
            path, node = [], 0
            while node is not None:
                path.append(node)
                said = best[first[b] + node]
                node = next((i for i, p in enumerate(par) if p == path[-1] and tok[i] == said), None)
            keep.append(path)
            texts[b] = torch.cat([texts[b], torch.tensor([tok[i] for i in path], device="cuda")])
            pending[b] = said
        most = max(map(len, keep))
        q.kv_compact(cache, pos, ints([p + [0] * (most - len(p)) for p in keep]), ints([len(p) for p in keep]))
        accepted.append([len(p) for p in keep])
    over_cache = model.step(pending, cache).float()
    texts = [torch.cat([t, p[None]]) for t, p in zip(texts, pending)]
    at_once = model.prompts(texts, new_cache(rows, cache_type)).float()
    return dict(accepted=accepted, lens=cache.lens.tolist(), texts=[len(t) for t in texts],
                status=int(cache.status), pages=int((cache.refs > 0).sum()), refs=int(cache.refs.sum()),
                difference=float((over_cache - at_once).norm() / at_once.norm()))


if __name__ == "__main__":
    for kind in (torch.float16, torch.float8_e4m3fn):
        r = main(cache_type=kind)
        print(f"cache of {kind}: tokens accepted per round and row:", r["accepted"])
        print("tokens in the rows:", r["lens"], "in", r["pages"], "pages")
        print(f"logits over the cache against one prompt: relative difference {r['difference']:.2e}")
